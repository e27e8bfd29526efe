"""The 4-bit attention's running maximum: phase 2 brings every weight to the last one by a power of two, so that a weight is rounded
to bf16 once, however large the logits are."""
import numpy as np
import pytest
import torch

from oracle import kv4_ops as K


def log2_scale():
    """A softmax scale that is 1 in log2 units, in fp32 as the library multiplies it."""
    s = np.float32(np.log(2))
    for _ in range(4):
        if s * np.float32(1.4426950408889634) == 1:
            return float(s)
        s = np.nextafter(s, np.float32(0))
    raise AssertionError("no such scale")


def test_scale_is_one_in_log2_units():
    assert np.float32(log2_scale()) * np.float32(1.4426950408889634) == np.float32(1)


@pytest.mark.gpu
@pytest.mark.parametrize("k,j", [(117, 46), (113, 46), (93, 46), (125, 46), (77, 46), (121, 37), (1, 64), (64, 37), (32, 100), (0, 0)])
@pytest.mark.parametrize("grow", [9, 10])
def test_weights_are_rounded_once_behind_a_growing_maximum(k, j, grow):
    """Logits of 2^17 and some 128ths (the distance of fp32 numbers there): 1,983 entries j / 128 below the first one, and one that
    lies `grow` - k / 128 above it, past 2^17, where the distance doubles.  Every key has 1 in one column, so the output there is
    Σ p / Σ p: off by a bf16 rounding of each p (2^-8), fp32 sums (n · 2^-24) and 2^x (2^-20)."""
    import sparse_attention_lightning_gb300 as dsa
    n, T = 31 * 64 + 1, 152  # an SM a query, so that a query's entries are one piece; the last entry has a chunk of its own
    logits = [2 ** 17 - 5 + k / 128] + [2 ** 17 - 5 + (k - j) / 128] * (n - 2) + [2 ** 17 - 5 + grow]
    bits = np.array([[int(z * 128) >> b & 1 for b in range(25)] for z in logits], float)  # 2^-7 .. 2^17
    lat = np.zeros((n + T, 512))
    lat[:, 500], lat[:, 511], lat[:, 16 * np.arange(31)] = 1, 6, 6  # 6 in every group of 16: its scale is 1
    for b in range(25):
        lat[:n, 16 * b + 1] = bits[:, b]
    rows = K.encode(lat, np.zeros((n + T, 64)))
    assert np.array_equal(K.decode(rows, 512, 64)[:, :512], lat)
    q = torch.zeros(T, 128, 576)
    for b in range(25):
        q[:, :, 16 * b + 1] = 2.0 ** (b - 7)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    P = dsa.Problem(i32([0, T]), i32([0, n + T]), q_lens=[T], k_lens=[n + T], h_idx=4, d_idx=32, h=128, d_c=512, d_rope=64, top_k=n,
                    idx_dtype="f32", kv_dtype="bf16", out_dtype="f32", sm_scale=log2_scale())
    idx = torch.arange(n, device="cuda", dtype=torch.int32).repeat(T, 1)
    out, lse = dsa.sparse_mla_attn4(P, q.bfloat16().cuda(), torch.from_numpy(rows).cuda(), idx)
    err = (out[:, :, 500].double() - 1).abs().max().item()
    assert err <= 2.0 ** -8 + n * 2.0 ** -24 + 2.0 ** -20, err * 256
    top = max(logits)
    want = (top + np.log2(sum(2.0 ** (z - top) for z in logits))) * np.log(2)
    assert (lse.double() - want).abs().max().item() <= 4 * 2.0 ** -24 * want
