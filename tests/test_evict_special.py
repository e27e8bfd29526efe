"""Eviction by weights that are not numbers, and from slices of wider rows."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import cache_ops as C
from sparse_attention_lightning_gb300 import _abi
from test_evict import _caches, _problem


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [[0x7FC00000], [0xFFC00000], [0x7FFFFFFF], [0xFFFFFFFF], [0x7F800001], [0xFF800001],
                                  [0xFFC00000, 0x7FC00000, 0x7F800001, 0xFFFFFFFF]])
@pytest.mark.parametrize("L,budget", [(300, 7), (300, 40), (2500, 900), (60000, 30)])
def test_every_nan_counts_as_largest(L, budget, bits):
    import sparse_attention_lightning_gb300 as dsa
    P, keys, caches, _ = _caches([L, 80], "e4m3", 0, seed=5, budget=budget)
    g = torch.Generator().manual_seed(L + budget)
    acc = torch.randn(2, L, generator=g)
    at = torch.randperm(L - 10, generator=g)[:20] + 3
    acc[0, at[10:]] = float("inf")
    acc[0, :2] = -float("inf")
    acc[0].view(torch.int32)[at[:10]] = torch.tensor(
        [b - (1 << 32) if b >> 31 else b for b in (bits * 10)[:10]], dtype=torch.int32)
    assert torch.isnan(acc[0]).sum() == 10
    r = dsa.evict(P, acc.cuda(), budget, 1, 2, kv=caches["kv"])
    a = acc[0].double().numpy()
    rank = np.where(np.isnan(a), 1e308, np.where(np.isinf(a), np.sign(a) * 1e300, a))
    want = C.keep(rank, budget, 1, 2)
    assert r.kept[0].tolist() == want.tolist()
    assert torch.equal(r.acc[0].cpu().view(torch.int32), acc[0][want].view(torch.int32))
    assert torch.equal(r.kv[:budget].cpu(), keys["kv"][want])


def test_acc_out_may_follow_a_strided_acc():
    """A slice of wider rows ends with its last element, not with its last row's stride."""
    L, A = _abi.lib(), 1 << 24
    p = _problem()  # 2 sequences, up to 40 positions

    def call(acc, ld, out, ld_out, budget=16):  # no workspace: the check behind this one refuses the call
        return L.dsa_evict(ctypes.byref(p), acc, ld, budget, 2, 4, 2 * A, 3 * A, out, ld_out, None, None, None, None, None,
                           None, None, 0, 0, 0, None, 1 << 30, None)

    bad, passed = _abi.DSA_ERR_INVALID_ARG, _abi.DSA_ERR_WORKSPACE
    assert call(A, 100, A + 4 * 140, 16) == passed and call(A, 100, A + 4 * 139, 16) == bad
    assert call(A + 4 * 66, 50, A, 50) == passed and call(A + 4 * 65, 50, A, 50) == bad
    assert call(A, 40, A + 4 * 80, 16) == passed and call(A, 40, A + 4 * 79, 16) == bad
