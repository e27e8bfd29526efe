"""Offsets that do not rise, in the 4-bit attention's forms for few queries: every kernel of a call takes a query for the same
sequence's, so that a row is either attended or left as it was."""
import numpy as np
import pytest
import torch

from oracle import cache_ops as C
from oracle import kv4_ops as K
from sparse_attention_lightning_gb300 import _abi


@pytest.mark.gpu
@pytest.mark.parametrize("top_k", [1500, 96])
@pytest.mark.parametrize("h", [128, 16])
def test_offsets_that_do_not_rise(h, top_k):
    """Queries 3 and 4 are sequence 0's by a search of the offsets and, by their values alone, also the inconsistent sequence 2's: they
    may be attended as the one or left as the other."""
    import sparse_attention_lightning_gb300 as dsa
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    g = torch.Generator().manual_seed(h)
    L = 1600
    P = dsa.Problem(i32([0, 5, 5, 8]), i32([0, L, L + 100, L + 102]), q_lens=[5, 0, 3], k_lens=[L, 100, 2], h_idx=4, d_idx=32, h=h,
                    d_c=512, d_rope=64, top_k=top_k, idx_dtype="f32", kv_dtype="bf16")
    rows = K.encode(torch.randn(L + 102, 512, generator=g).double().numpy(), torch.randn(L + 102, 64, generator=g).numpy())
    q = torch.randn(8, h, 576, generator=g).bfloat16()
    idx = torch.stack([torch.randperm(L - 8, generator=g)[:top_k] for _ in range(8)]).to(torch.int32)
    P.cu_q.copy_(i32([0, 5, 3, 8]))  # sequence 2: five queries of two positions
    ws = dsa.Workspace(nbytes=P.workspace_size(_abi.OP_SPARSE_MLA_ATTN4))
    ws.buf[_abi.STATUS_BYTES:] = 0x55
    out, lse = torch.full((8, h, 512), 7.0, device="cuda").bfloat16(), torch.full((8, h), 7.0, device="cuda")
    dsa.sparse_mla_attn4(P, q.cuda(), torch.from_numpy(rows).cuda(), idx.cuda(), out=out, lse=lse, ws=ws)
    assert ws.status() == _abi.DSA_FLAG_BAD_SEQS
    assert (out[5:] == 7).all() and (lse[5:] == 7).all()
    keys = K.decode(rows, 512, 64)
    assert not (out[:3] == 7).all(dim=2).any()
    for t in range(5):
        if (out[t] == 7).all() and (lse[t] == 7).all():
            continue
        ro, rl, mag, top = C.attend(q[t].double().numpy(), keys[idx[t].numpy()], 512, P.scale)
        delta = 578 * 2.0 ** -24 * top  # as in the other tests of this attention: logits, fp32 sums, 2^x, P and output in bf16
        rel = 2 * delta + top_k * 2.0 ** -24 + 2.0 ** -20
        err = np.abs(out[t].double().cpu().numpy() - ro)
        assert np.all(err <= (rel[:, None] + 2.0 ** -8) * mag * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ro) + 1e-38), t
        bound = delta + (top_k + 8) * 2.0 ** -24 + 2.0 ** -20 * (1 + np.abs(rl))
        assert np.all(np.abs(lse[t].double().cpu().numpy() - rl) <= bound), t
