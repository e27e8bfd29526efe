"""The 4-bit attention's queries on the tensor cores: a latent column is off by at most 2^-39 of the head's largest, also where no key
has anything in the largest one's column, so that the small ones alone decide."""
import numpy as np
import pytest
import torch

from oracle import cache_ops as C
from oracle import kv4_ops as K


@pytest.mark.gpu
@pytest.mark.parametrize("h", [128, 16])
def test_columns_far_below_the_largest(h):
    import sparse_attention_lightning_gb300 as dsa
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    g = torch.Generator().manual_seed(h)
    n = 130
    P = dsa.Problem(i32([0, 1]), i32([0, n]), q_lens=[1], k_lens=[n], h_idx=4, d_idx=32, h=h, d_c=512, d_rope=64, top_k=n,
                    idx_dtype="f32", kv_dtype="bf16", out_dtype="f32")
    lat = torch.randn(n, 512, generator=g).double().numpy()
    lat[:, 0] = 0
    rows = K.encode(lat, np.zeros((n, 64)))
    keys = K.decode(rows, 512, 64)
    assert (keys[:, 0] == 0).all()
    q = torch.randn(1, h, 576, generator=g) * 3
    far = torch.tensor([10, 24, 27, 29, 31, 33, 36, 38, 41, 45])[torch.arange(h) % 10]
    q[0, :, 0] = 2.0 ** far
    q = q.bfloat16()
    idx = torch.arange(n, dtype=torch.int32)[None]
    out, lse = dsa.sparse_mla_attn4(P, q.cuda(), torch.from_numpy(rows).cuda(), idx.cuda())
    ro, rl, mag, top = C.attend(q[0].double().numpy(), keys, 512, P.scale)
    lost = 2.0 ** -39 * 2.0 ** far.double().numpy() * P.scale * np.abs(keys[:, 1:512]).sum(axis=1).max()  # of a logit
    delta = 578 * 2.0 ** -24 * top + lost
    rel = np.expm1(np.minimum(2 * delta, 100)) + n * 2.0 ** -24 + 2.0 ** -20  # (infinity times a column of zeros would be no bound)
    err = np.abs(out[0].double().cpu().numpy() - ro)
    assert np.all(err <= (rel[:, None] + 2.0 ** -8) * mag * (1 + 2.0 ** -24) + 2.0 ** -24 * np.abs(ro) + 1e-38)
    assert np.all(np.abs(lse[0].double().cpu().numpy() - rl) <= delta + (n + 8) * 2.0 ** -24 + 2.0 ** -20 * (1 + np.abs(rl)))
