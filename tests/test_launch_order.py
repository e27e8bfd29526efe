"""What programmatic dependent launches are ordered by: a kernel that such a launch may start beside the one before it lets the next
one start only behind its own wait, as the next one may read, ahead of its wait, what the one before both has written."""
import glob
import os
import re

import pytest
import torch

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_attention_lightning_gb300", "csrc")


def kernels():
    """(file, kernel, body) of every kernel."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        with open(path) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        for m in re.finditer(r"__global__[^;{]*?\b(\w+_kernel)\s*\(", text):
            start = text.index("{", m.end())
            depth, end = 0, start
            while True:  # the matching brace
                depth += {"{": 1, "}": -1}.get(text[end], 0)
                end += 1
                if depth == 0:
                    break
            yield os.path.basename(path), m.group(1), text[start:end], text


# The kernel in front of it is its own operator's, launched plainly, and clears what this one adds to.
BEHIND_OWN = {"attn_weights_tc_kernel"}


def test_next_kernels_are_released_behind_the_wait():
    seen = set()
    for file, name, body, text in kernels():
        launch = body.find("griddep_launch()")
        if launch < 0 or name in BEHIND_OWN:
            continue
        plain = re.search(rf"\b(kern|{name})\b[^;]*<<<", text) or "cudaLaunchAttributeCooperative" in text
        if "launch_pdl(" not in text or (plain and "griddep_wait()" not in body):
            continue  # it starts behind the kernel before it as a whole
        wait = body.find("griddep_wait()")
        assert 0 <= wait < launch, f"{file}: {name} lets the next kernel start ahead of its own wait"
        seen.add(name)
    assert {"attn4_tc_kernel", "attn4_simt_kernel", "reserve_kernel", "compact_kernel", "prefix_tc_kernel", "prefix_simt_kernel",
            "topk_stream_kernel", "evict_select_kernel"} <= seen


@pytest.mark.gpu
@pytest.mark.parametrize("queries,top_k", [(1, 2048), (3, 512), (2, 2048)])
def test_what_was_written_before_a_call_is_what_the_next_call_reads(queries, top_k):
    """Offsets and queries written in place, attention over the 4-bit cache (in pieces that a merge joins), attention over it and over
    the bf16 cache again, many times over without a synchronisation, against the same calls one by one."""
    import sparse_attention_lightning_gb300 as dsa
    g = torch.Generator(device="cuda").manual_seed(queries)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    L, h = 4096, 128
    P = dsa.Problem(i32([0, queries]), i32([0, L]), q_lens=[queries], k_lens=[L], h_idx=4, d_idx=32, h=h, d_c=512, d_rope=64,
                    top_k=top_k, idx_dtype="f32", kv_dtype="bf16")
    kv = torch.randn(L, 576, generator=g, device="cuda").bfloat16()
    # the new tokens are sequence 0's last ones, so writing takes a problem in which all tokens are new
    A = dsa.Problem(i32([0, L]), i32([0, L]), q_lens=[L], k_lens=[L], h_idx=4, d_idx=32, h=h, d_c=512, d_rope=64, top_k=1,
                    idx_dtype="f32", kv_dtype="bf16")
    kv4 = torch.zeros(L, dsa.kv4_row_bytes(512, 64), dtype=torch.uint8, device="cuda")
    dsa.write_kv4(A, kv[:, :512], kv[:, 512:], kv4)
    idx = torch.stack([torch.randperm(L - queries, generator=g, device="cuda")[:top_k] for _ in range(queries)]).to(torch.int32)
    qs = [torch.randn(queries, h, 576, generator=g, device="cuda").bfloat16() for _ in range(3)]
    cu = P.cu_q.clone()
    q, ws = torch.zeros_like(qs[0]), dsa.Workspace()
    rot = dsa.Rotary(64)
    pos = torch.arange(queries, device="cuda", dtype=torch.int32)

    def step(i, sync):
        P.cu_q.copy_(cu)
        q.copy_(qs[i % 3])
        dsa.rotate_axes(q[..., 512:], pos + i % 5, rot, out=q[..., 512:])
        got = [*dsa.sparse_mla_attn4(P, q, kv4, idx, ws=ws)]
        if sync:
            torch.cuda.synchronize()
        got += dsa.sparse_mla_attn4(P, q, kv4, idx, ws=ws)
        if sync:
            torch.cuda.synchronize()
        got += dsa.sparse_mla_attn(P, q, kv, idx, ws=ws)
        q.zero_()
        P.cu_q.zero_()  # (offsets of no query, for whoever reads them late)
        return got

    want = [step(i, True) for i in range(15)]
    torch.cuda.synchronize()
    got = [step(i, False) for i in range(60)]
    assert ws.status() == 0
    for i in range(60):
        assert all(torch.equal(a, b) for a, b in zip(got[i], want[i % 15])), i
