"""Rotary positions with several axes (dsa_rotate_axes) against the fp64 definition."""
import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import kv4_ops as K
from sparse_attention_lightning_gb300 import _abi

BF, F32 = torch.bfloat16, torch.float32


def test_oracle_rotates_pairs():
    x = np.array([[3.0, 4.0, 1.0, 0.0]])
    y = K.rotate(x, np.array([[math.pi / 2, math.pi]]), True)
    assert np.allclose(y, [[-4, 3, -1, 0]])
    y = K.rotate(x, np.array([[math.pi / 2, math.pi]]), False)
    assert np.allclose(y, [[-1, -4, 3, 0]])


def test_turns_are_fractions_of_2_64():
    import sparse_attention_lightning_gb300 as dsa
    r = dsa.Rotary(8, inv_freq=[2 * math.pi, math.pi, math.pi / 2, -math.pi / 2])
    assert list(r.turn) == [0, 1 << 63, 1 << 62, 3 << 62]
    r = dsa.Rotary(64, sections=[16, 8, 8])
    assert list(r.axis) == [0] * 16 + [1] * 8 + [2] * 8 and r.num_axes == 3
    f = 10000.0 ** (-5 / 32)
    assert abs(r.turn[5] / 2.0 ** 64 - f / (2 * math.pi)) <= 2.0 ** -53
    for bad in (dict(d_rope=7), dict(d_rope=0), dict(d_rope=258), dict(d_rope=8, sections=[3]),
                dict(d_rope=8, sections=[5, -1]), dict(d_rope=8, sections=[4], axes=[0] * 4),
                dict(d_rope=8, inv_freq=[1.0] * 3), dict(d_rope=8, inv_freq=[1.0, 1.0, 1.0, float("inf")]),
                dict(d_rope=8, axes=[0, 0, -1, 0]), dict(d_rope=8, axes=[0, 0, 255, 0])):
        with pytest.raises(ValueError):
            dsa.Rotary(**bad)


def test_argument_checks():
    L, A = _abi.lib(), 1 << 20
    bad, unsup = _abi.DSA_ERR_INVALID_ARG, _abi.DSA_ERR_UNSUPPORTED
    turn, axis = (ctypes.c_uint64 * 128)(), (ctypes.c_uint8 * 128)()

    def call(T=4, H=2, d=64, dt=1, axes=1, turn=turn, axis=axis, pos=1 << 30, ld=4, x=A, xt=128, xh=64, out=1 << 24,
             ot=128, oh=64):
        return L.dsa_rotate_axes(T, H, d, dt, 1, 0, axes, turn, axis, pos, ld, x, xt, xh, out, ot, oh, None)

    assert call(T=-1) == bad and call(H=0) == bad and call(dt=2) == bad and call(axes=0) == bad and call(axes=256) == bad
    assert call(d=63) == unsup and call(d=0) == unsup and call(d=258) == unsup
    assert call(ld=3) == bad and call(ld=-1) == bad and call(turn=None) == bad and call(axis=None) == bad
    assert call(axis=(ctypes.c_uint8 * 128)(0, 1)) == bad          # an axis without positions
    assert call(x=None) == bad and call(out=None) == bad and call(x=A + 1) == bad and call(pos=None) == bad
    assert call(pos=(1 << 30) + 2) == bad and call(xt=-1) == bad and call(oh=-64) == bad
    assert call(oh=63) == bad and call(ot=127) == bad              # rows of out that share columns
    assert call(out=A + 64) == bad                                 # shifted by half a row
    assert call(out=A, ot=256) == bad                              # in place, other strides
    assert call(out=A + 128 * 2, xt=512, ot=512, xh=128, oh=128) == bad  # another head of the same tensor
    assert call(out=(1 << 30) - 8) == bad                          # the positions
    assert call(T=0, x=None, out=None, pos=None, ld=0) == _abi.DSA_OK


def reference(x, pos, freq, axis, interleaved, inverse):
    x = x.double().numpy()
    angle = pos.double().numpy()[axis].T * np.array(freq)  # [T, pairs]
    angle = -angle if inverse else angle
    angle = angle[:, None] if x.ndim == 3 else angle
    d = x.shape[-1]
    u, v = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :d // 2], x[..., d // 2:])
    r = np.abs(u) + np.abs(v)
    mag = np.empty_like(x)
    if interleaved:
        mag[..., 0::2] = mag[..., 1::2] = r
    else:
        mag[..., :d // 2] = mag[..., d // 2:] = r
    return K.rotate(x, angle, interleaved), mag


def check(y, x, pos, freq, axis, interleaved, inverse=False):
    """The angle is off by 2^-25 half turns (an fp32 number below 1), so by less than 2^-23; sine and cosine by 2 units,
    2^-22 together with the angle's; two products and their sum by 2^-24 each of |u| + |v|: 2^-20 in all is over twice
    that.  Both this reference's angles and the fixed-point turns go by f rounded to 53 bits: 2^-51 of the
    position.  The output is rounded once."""
    ref, mag = reference(x, pos, freq, axis, interleaved, inverse)
    far = float(pos.double().abs().max()) * 2.0 ** -51 if pos.numel() else 0.0
    half = 2.0 ** -8 if y.dtype == BF else 2.0 ** -24
    err = np.abs(y.double().cpu().numpy() - ref)
    assert np.all(err <= (2.0 ** -20 + far) * (1 + half) * mag + half * np.abs(ref) + 1e-38), err.max()


CASES = [
    # T, H, d, width of the tensor, axes, interleaved
    (1, 128, 64, 576, 3, True), (1, 1, 64, 64, 1, False), (5, 3, 16, 32, 2, True), (7, 20, 48, 48, 3, False),
    (33, 128, 64, 576, 3, False), (301, 16, 128, 640, 4, True), (2, 5, 2, 2, 1, True), (3, 7, 6, 9, 2, False),
    (4, 9, 10, 17, 2, True), (2, 3, 256, 256, 3, False), (600, 64, 64, 576, 3, True), (700, 64, 64, 576, 3, False),
    (2500, 8, 64, 64, 2, True), (130, 130, 32, 40, 3, True),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,H,d,width,axes,interleaved", CASES)
def test_values(T, H, d, width, axes, interleaved, dtype):
    import sparse_attention_lightning_gb300 as dsa
    g = torch.Generator().manual_seed(T + d)
    x = torch.randn(T, H, width, generator=g).to(dtype)
    pos = torch.randint(-(1 << 20), 1 << 20, (axes, T), generator=g, dtype=torch.int32)
    n = d // 2
    axis = [i * axes // n for i in range(n)]
    rot = dsa.Rotary(d, axes=axis, interleaved=interleaved)
    freq = [10000.0 ** (-i / n) for i in range(n)]
    pos = pos[:rot.num_axes]
    whole = x.cuda()
    part = whole[..., width - d:]
    y = dsa.rotate_axes(part, pos.cuda(), rot)
    check(y, x[..., width - d:], pos, freq, axis, interleaved)
    z = dsa.rotate_axes(part, pos.cuda(), rot, inverse=True)
    check(z, x[..., width - d:], pos, freq, axis, interleaved, inverse=True)
    # in place: the same bytes, and the other columns stay
    got = dsa.rotate_axes(part, pos.cuda(), rot, out=part)
    assert got is part and torch.equal(part, y) and torch.equal(whole[..., :width - d].cpu(), x[..., :width - d])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
def test_layouts(dtype):
    """Keys without heads, transposed heads, unaligned slices, a column range of the same tensor, broadcast heads."""
    import sparse_attention_lightning_gb300 as dsa
    g = torch.Generator().manual_seed(1)
    rot = dsa.Rotary(16, sections=[5, 3], interleaved=False)
    freq = [10000.0 ** (-i / 8) for i in range(8)]
    args = (freq, [0] * 5 + [1] * 3, False)
    pos = torch.randint(0, 9999, (2, 37), generator=g, dtype=torch.int32)
    wide = torch.randint(0, 9999, (3, 50), generator=g, dtype=torch.int32)
    wide[:2, :37] = pos
    strided = wide.cuda()[:2, :37]
    x = torch.randn(37, 40, generator=g).to(dtype)
    for at in (0, 8, 3):  # a key's rope columns, aligned and not
        y = dsa.rotate_axes(x.cuda()[:, at:at + 16], strided, rot)
        assert y.shape == (37, 16) and y.is_contiguous()
        check(y, x[:, at:at + 16], pos, *args)
    x = torch.randn(6, 37, 16, generator=g).to(dtype)  # heads first
    dev = x.cuda()
    y = dsa.rotate_axes(dev.transpose(0, 1), strided, rot, out=torch.empty_like(dev).transpose(0, 1))
    check(y, x.transpose(0, 1), pos, *args)
    x = torch.randn(37, 6, 48, generator=g).to(dtype)
    dev = x.cuda()
    y = dsa.rotate_axes(dev[..., 32:], strided, rot, out=dev[..., :16])
    check(y, x[..., 32:], pos, *args)
    assert torch.equal(dev[..., 16:].cpu(), x[..., 16:])
    x = torch.randn(37, 1, 16, generator=g).to(dtype)
    y = dsa.rotate_axes(x.cuda().expand(37, 5, 16), strided, rot)
    check(y, x.expand(37, 5, 16), pos, *args)
    same = pos[:1].expand(2, 37)  # text: every axis has the token's position
    y = dsa.rotate_axes(x.cuda(), pos[:1].cuda().expand(2, 37), rot)
    check(y, x, same, *args)


@pytest.mark.gpu
def test_far_positions_and_whole_turns():
    import sparse_attention_lightning_gb300 as dsa
    x = torch.randn(4, 2, 8, generator=torch.Generator().manual_seed(2))
    freq = [1.0, 0.37, 10000.0 ** -0.5, 1e-4]
    pos = torch.tensor([[2147483647, -2147483648, 0, 1]], dtype=torch.int32)
    y = dsa.rotate_axes(x.cuda(), pos.cuda(), dsa.Rotary(8, inv_freq=freq))
    check(y, x, pos, freq, [0] * 4, True)
    # turns of a half, a quarter and whole ones are exact, at any position
    quarter = dsa.Rotary(8, inv_freq=[2 * math.pi, math.pi, math.pi / 2, 6 * math.pi])
    y = dsa.rotate_axes(x.cuda(), torch.tensor([5, -3, 0, 2147483647], dtype=torch.int32).cuda(), quarter).cpu()
    assert torch.equal(y[..., :2], x[..., :2]) and torch.equal(y[..., 6:], x[..., 6:])
    assert torch.equal(y[0, :, 2:4], -x[0, :, 2:4]) and torch.equal(y[2], x[2])
    assert torch.equal(y[0, :, 4], -x[0, :, 5]) and torch.equal(y[0, :, 5], x[0, :, 4])


@pytest.mark.gpu
def test_special_values_stay_in_their_pair():
    import sparse_attention_lightning_gb300 as dsa
    x = torch.randn(3, 2, 16, generator=torch.Generator().manual_seed(3))
    x[1, 1, 4], x[2, 0, 9] = float("nan"), float("inf")
    pos = torch.tensor([7, 8, 9], dtype=torch.int32)
    y = dsa.rotate_axes(x.cuda(), pos.cuda(), dsa.Rotary(16)).cpu()
    odd = ~torch.isfinite(y)
    want = torch.zeros_like(odd)
    want[1, 1, 4:6] = want[2, 0, 8:10] = True
    assert torch.equal(odd, want)


@pytest.mark.gpu
def test_empty_streams_graphs_and_refusals():
    import sparse_attention_lightning_gb300 as dsa
    rot = dsa.Rotary(64, sections=[16, 8, 8])
    pos = torch.arange(30, dtype=torch.int32).reshape(3, 10).cuda()
    assert dsa.rotate_axes(torch.empty(0, 4, 64).cuda(), pos[:, :0], rot).shape == (0, 4, 64)
    assert dsa.rotate_axes(torch.empty(10, 0, 64).cuda(), pos, rot).shape == (10, 0, 64)
    x = torch.randn(10, 4, 64, generator=torch.Generator().manual_seed(4)).cuda()
    want = dsa.rotate_axes(x, pos, rot)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = dsa.rotate_axes(x, pos, rot)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    graph, y = torch.cuda.CUDAGraph(), torch.empty_like(x)
    with torch.cuda.graph(graph, stream=side):
        dsa.rotate_axes(x, pos, rot, out=y)
    for _ in range(2):
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
    for bad in (lambda: dsa.rotate_axes(x.cpu(), pos, rot), lambda: dsa.rotate_axes(x.half(), pos, rot),
                lambda: dsa.rotate_axes(x, pos[:2], rot), lambda: dsa.rotate_axes(x, pos.long(), rot),
                lambda: dsa.rotate_axes(x, pos.cpu(), rot), lambda: dsa.rotate_axes(x[..., :32], pos, rot),
                lambda: dsa.rotate_axes(x, pos, rot, out=y[:9]), lambda: dsa.rotate_axes(x, pos, rot, out=y.bfloat16()),
                lambda: dsa.rotate_axes(x[0, 0], pos, rot), lambda: dsa.rotate_axes(x.transpose(1, 2), pos, rot),
                lambda: dsa.rotate_axes(x, pos.t().contiguous().t(), rot)):
        with pytest.raises(ValueError):
            bad()
    wide = torch.zeros(11, 4, 64).cuda()
    with pytest.raises(dsa.DsaError):
        dsa.rotate_axes(wide[:10], pos, rot, out=wide[1:])
    with pytest.raises(dsa.DsaError):
        dsa.rotate_axes(x, pos, rot, out=x[:, :1].expand(10, 4, 64))
