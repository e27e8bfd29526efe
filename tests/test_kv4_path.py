"""Which kernel attends over the 4-bit cache: the tensor-core kernel for 512 + 64 bf16 columns wherever the build's registers
suffice for its roles, and never a refusal for how it was built."""
import os
import re

import pytest
import torch

PKG = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_attention_lightning_gb300")


def test_a_build_is_not_refused():
    with open(os.path.join(PKG, "csrc", "attn4_tc.cu")) as f:
        text = f.read()
    assert not re.search(r"DSA_ERR_UNSUPPORTED[^;]*built", text)
    eligible = re.search(r"bool attn4_tc_eligible\([^}]*\}", text).group(0)
    assert "built_to_run()" in eligible  # the other kernel serves it


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,dims,kernel", [("bf16", (512, 64), "attn4_tc"), ("bf16", (256, 32), "attn4_simt"),
                                               ("f32", (512, 64), "attn4_simt")])
def test_kernel_of_a_width(dtype, dims, kernel):
    import sparse_attention_lightning_gb300 as dsa
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    P = dsa.Problem(i32([0, 2]), i32([0, 90]), q_lens=[2], k_lens=[90], h_idx=4, d_idx=32, h=128, d_c=dims[0], d_rope=dims[1],
                    top_k=64, idx_dtype="f32", kv_dtype=dtype)
    q = torch.randn(2, 128, sum(dims), device="cuda").to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    kv4 = torch.zeros(90, dsa.kv4_row_bytes(*dims), dtype=torch.uint8, device="cuda")
    idx = torch.arange(64, device="cuda", dtype=torch.int32).repeat(2, 1)
    with dsa.trace() as t:
        dsa.sparse_mla_attn4(P, q, kv4, idx)
    names = {name for name, _ in t.records}
    assert kernel in names and len({n for n in names if n.startswith("attn4")}) == 1


@pytest.mark.gpu
@pytest.mark.parametrize("queries,h,top_k,merged", [
    (1, 128, 2048, True), (12, 128, 2048, True), (18, 128, 2048, True), (32, 128, 2048, False), (64, 128, 2048, False),
    (152, 128, 2048, False), (4, 16, 2048, True), (18, 16, 2048, True), (48, 16, 2048, True), (64, 16, 2048, False), (2, 128, 512, True),
    (36, 128, 512, False), (12, 64, 2048, True), (30, 64, 2048, False)])
def test_form_for_few_queries(queries, h, top_k, merged):
    """Partial outputs and a merge, or clusters, as measured at these sizes (each at least 2 % apart)."""
    import sparse_attention_lightning_gb300 as dsa
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    L = 2048 + queries
    P = dsa.Problem(i32([0, queries]), i32([0, L]), q_lens=[queries], k_lens=[L], h_idx=4, d_idx=32, h=h, d_c=512, d_rope=64,
                    top_k=top_k, idx_dtype="f32", kv_dtype="bf16")
    q = torch.randn(queries, h, 576, device="cuda").bfloat16()
    kv4 = torch.zeros(L, 416, dtype=torch.uint8, device="cuda")
    idx = torch.arange(top_k, device="cuda", dtype=torch.int32).repeat(queries, 1)
    with dsa.trace() as t:
        out, lse = dsa.sparse_mla_attn4(P, q, kv4, idx)
    assert any("merge" in name for name, _ in t.records) == merged
    assert (out == 0).all() and torch.allclose(lse, torch.full_like(lse, top_k).log(), rtol=0, atol=1e-4)
