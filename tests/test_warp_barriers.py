"""Barrier instructions that a warp executes as one (.aligned) stand behind a __syncwarp(): lanes that come apart out of a role's
loop would otherwise be counted at two barriers."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_attention_lightning_gb300", "csrc")


def test_aligned_barriers_reconverge_the_warp_first():
    found = 0
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        with open(path) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        for m in re.finditer(r'asm\s+volatile\s*\(\s*"barrier\.[a-z.]*aligned', text):
            found += 1
            before = text[:m.start()].rstrip()
            assert before.endswith("__syncwarp();"), f"{os.path.basename(path)}: {text[m.start():m.start() + 70]}"
    assert found >= 5
