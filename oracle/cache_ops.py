"""The operators around the caches in fp64 numpy, one row or one sequence at a time, written from
their definitions.

The code shares nothing with the CUDA path.  Inputs are float64 (the exact values the kernels' bf16
or fp32 inputs hold).
"""
from __future__ import annotations

import numpy as np


def rmsnorm(x, w, residual=None, eps=1e-6):
    """(y, h) of rows x [R, d]: h = x + residual, y = h / sqrt(mean h² + eps) · w."""
    h = x if residual is None else x + residual
    return h / np.sqrt((h * h).mean(axis=1, keepdims=True) + eps) * w, h


def e4m3_scale(y):
    """amax / 448 of each row, 1 where that is no normal fp32 number."""
    s = np.abs(y).max(axis=1) / 448.0
    return np.where(s < 2.0 ** -126, 1.0, s)


def mx_exponent(y):
    """The smallest e (from -127) with amax <= 448 · 2^e over 32 elements, 0 for zeros: [R, d/32]."""
    a = np.abs(y.reshape(y.shape[0], -1, 32)).max(axis=2)
    e = np.ceil(np.log2(np.where(a > 0, a, 448.0) / 448.0)).astype(int)
    return np.maximum(e, -127)


def attend(q, keys, d_c, scale):
    """Dense attention of q [H, D] over keys [n, D]: (out [H, d_c], lse [H], Σ p|v| [H, d_c],
    max Σ_c |q_c k_c| · scale [H]).  The last two bound rounding errors.  n = 0: zeros and -inf."""
    H = q.shape[0]
    if keys.shape[0] == 0:
        return np.zeros((H, d_c)), np.full(H, -np.inf), np.zeros((H, d_c)), np.zeros(H)
    S = q @ keys.T * scale
    m = S.max(axis=1, keepdims=True)
    p = np.exp(S - m)
    l = p.sum(axis=1, keepdims=True)
    p /= l
    mag = (np.abs(q) @ np.abs(keys).T).max(axis=1) * scale
    return p @ keys[:, :d_c], (m + np.log(l))[:, 0], p @ np.abs(keys[:, :d_c]), mag


def weights(q, keys, lse, scale):
    """Σ_h exp(scale q_h·key − lse_h) of each key, heads with lse = -inf left out: [n]."""
    live = np.isfinite(lse)
    return np.exp(q[live] @ keys.T * scale - lse[live, None]).sum(axis=0)


def keep(acc, budget, sink, recent):
    """Positions to keep of a sequence with accumulated weights acc [L], ascending."""
    L = acc.shape[0]
    if L <= budget:
        return np.arange(L)
    mid = np.arange(sink, L - recent)
    best = mid[np.argsort(-acc[mid], kind="stable")[:budget - sink - recent]]
    return np.sort(np.concatenate([np.arange(sink), best, np.arange(L - recent, L)]))
