"""Rotated columns written beside their source in one tensor: allowed wherever no row of out shares an element with a row of x, in any
order of tokens and heads, and refused wherever one does."""
import ctypes
import random

import pytest
import torch

from sparse_attention_lightning_gb300 import _abi


def test_heads_outside_tokens_and_tokens_of_more_than_their_heads():
    """Calls of so many rows that they are refused for it, behind the checks of overlaps: DSA_ERR_UNSUPPORTED."""
    L, A = _abi.lib(), 1 << 20
    bad, unsup = _abi.DSA_ERR_INVALID_ARG, _abi.DSA_ERR_UNSUPPORTED
    T, H = 1 << 30, 1 << 9
    turn, axis = (ctypes.c_uint64 * 1)(), (ctypes.c_uint8 * 1)()

    def call(off, st, sh):
        return L.dsa_rotate_axes(T, H, 2, _abi.DSA_BF16, 1, 0, 1, turn, axis, 1 << 46, T, A, st, sh, A + 2 * off, st, sh, None)

    for st, sh in ((4, 4 * T), (4 * H, 4), (4 * H + 6, 4), (6, 6 * T + 2)):  # [H, T, ...], [T, H, ...], and with more behind a row's heads
        assert call(2, st, sh) == unsup
        assert call(1, st, sh) == bad and call(max(st, sh), st, sh) == bad and call(-1, st, sh) == bad
    # between the columns of the next token, which begin 6 behind the last head; one column into them
    assert call(4 * H + 4, 4 * H + 6, 4) == unsup and call(4 * H + 5, 4 * H + 6, 4) == bad


@pytest.mark.gpu
@pytest.mark.parametrize("seed", range(4))
def test_every_shift_within_one_tensor(seed):
    import sparse_attention_lightning_gb300 as dsa
    r = random.Random(seed)
    ran = refused = 0
    for _ in range(60):
        d, T, H = r.choice((2, 4, 8)), r.randint(1, 4), r.randint(1, 4)
        inner = d + r.choice((0, 0, 2, 3, d, d + 1))
        if r.random() < 0.5:
            sh, st = inner, inner * H + r.choice((0, 0, 5, 2 * d))
        else:
            st, sh = inner, inner * T + r.choice((0, 0, 5, 2 * d))
        span = (T - 1) * st + (H - 1) * sh + d
        off = r.randint(-span - 1, span + 1)
        buf = torch.randn(3 * span + 4, generator=torch.Generator().manual_seed(seed)).cuda()
        view = lambda o: buf.as_strided((T, H, d), (st, sh, 1), o)  # noqa: E731
        at = lambda o: {o + t * st + h * sh + c for t in range(T) for h in range(H) for c in range(d)}  # noqa: E731
        first = span + 1
        x, out = view(first), view(first + off)
        pos = torch.arange(1, T + 1, dtype=torch.int32).cuda()
        rot, before = dsa.Rotary(d), buf.clone()
        if off and at(first) & at(first + off):
            with pytest.raises(dsa.DsaError):
                dsa.rotate_axes(x, pos, rot, out=out)
            assert torch.equal(buf, before)
            refused += 1
            continue
        want = dsa.rotate_axes(x.contiguous(), pos, rot)
        dsa.rotate_axes(x, pos, rot, out=out)
        assert torch.equal(out, want)
        rest = sorted(set(range(buf.numel())) - at(first + off))
        assert torch.equal(buf[rest], before[rest])
        ran += 1
    assert ran >= 5 and refused >= 5  # (the draws hold both)
