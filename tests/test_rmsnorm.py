"""Residual addition, RMS norm and 8-bit output (dsa_add_rmsnorm) against the fp64 definition."""
import numpy as np
import pytest
import torch

from oracle import cache_ops as C
from oracle.dsa_oracle import e4m3_to_f64
from sparse_attention_lightning_gb300 import _abi

EPS = 1e-6


def test_oracle_closed_forms():
    y, h = C.rmsnorm(np.array([[3.0, -4.0]]), np.array([1.0, 2.0]), np.array([[0.0, 8.0]]), 0.0)
    assert np.allclose(h, [[3.0, 4.0]]) and np.allclose(y, [[3 / 12.5 ** 0.5, 8 / 12.5 ** 0.5]])
    g = np.zeros((1, 128))
    g[0, 0], g[0, 40], g[0, 70] = 448.0, -448.5, 2.0 ** -150
    assert C.mx_exponent(g).tolist() == [[0, 1, -127, 0]]
    assert C.e4m3_scale(np.array([[0.0, 0.0], [896.0, 1.0]])).tolist() == [1.0, 2.0]


def test_argument_checks():
    L = _abi.lib()
    A = 1 << 20  # never dereferenced: every check fails first

    def call(rows=4, d=64, dtype=1, quant=0, eps=EPS, x=A, ld=64, res=None, ldr=64, w=2 * A,
             h=None, y=3 * A, codes=None, scale=None):
        return L.dsa_add_rmsnorm(rows, d, dtype, quant, eps, x, ld, res, ldr, w, h, y, codes, scale,
                                 None)

    bad, unsup = _abi.DSA_ERR_INVALID_ARG, _abi.DSA_ERR_UNSUPPORTED
    assert call(rows=0, x=None, w=None, y=None) == _abi.DSA_OK
    assert call(rows=-1) == bad and call(d=0) == bad and call(dtype=2) == unsup
    assert call(quant=1) == bad and call(eps=-1.0) == bad and call(eps=float("nan")) == bad
    assert call(x=None) == bad and call(y=None) == bad and call(w=None) == bad
    assert call(ld=63) == bad and call(x=A + 1) == bad and call(rows=1 << 31) == unsup
    assert call(res=4 * A) == bad and call(h=4 * A) == bad                # one without the other
    assert call(quant=2, y=None, codes=5 * A) == bad                      # no scale
    assert call(quant=3, d=48, ld=48, codes=5 * A, scale=6 * A) == unsup  # not whole groups
    assert call(y=A + 128) == bad                       # y over the next row of x
    assert call(x=A, ld=128, y=A) == bad                # in place, but x's rows are apart
    assert call(res=4 * A, h=3 * A) == bad              # h_out is y
    assert call(quant=2, codes=A, scale=6 * A) == bad   # codes over x
    assert call(quant=2, y=None, codes=5 * A, scale=6 * A + 2) == bad


def _close(got, ref, rel, what):
    err = np.abs(got - ref)
    assert np.all(err <= rel * np.abs(ref) + 1e-30), (what, float((err / (np.abs(ref) + 1e-30)).max()))


def _check(x, w, res, eps, quant, y, h, codes, scale):
    """Errors counted: Σ h² is added in chains of at most max(64, d / 1024 + 16) fp32 additions (relative error
    below that many 2^-24; half of it in the square root), then six more roundings; a result stored
    in type t is off by eps(t) / 2 more.  E4M3 codes: half a step, 2^-4 relative or 2^-10 absolute
    in units of the scale."""
    d = x.shape[1]
    f64 = lambda t: t.cpu().double().numpy()  # noqa: E731
    ry, rh = C.rmsnorm(f64(x), f64(w), None if res is None else f64(res), eps)
    rel = (max(64, d / 1024 + 16) / 2 + 6) * 2.0 ** -24
    half = torch.finfo(x.dtype).eps / 2
    if res is not None:
        # h is exact in fp32 up to one rounding, and rounded once more for bf16
        assert torch.equal(h.cpu(), (x.cpu().float() + res.cpu().float()).to(x.dtype))
        # the sum's own rounding (2^-24 of h) reaches y where h cancels: bounded by the norm's scale
        rel += 2.0 ** -24
    if y is not None:
        _close(f64(y), ry, rel + half * (1 + rel), "y")
    if quant == "e4m3":
        s = f64(scale).reshape(-1)
        _close(s, C.e4m3_scale(ry), rel + 2.0 ** -22, "scale")
        v = e4m3_to_f64(codes.cpu().numpy()) * s[:, None]
        tol = np.maximum(np.abs(ry) * 2.0 ** -4, s[:, None] * 2.0 ** -10)
        assert np.all(np.abs(v - ry) <= tol * (1 + 2.0 ** -10))
    elif quant == "mxfp8":
        e = scale.cpu().numpy().astype(int) - 127
        top = np.abs(ry.reshape(ry.shape[0], -1, 32)).max(axis=2)
        ref = C.mx_exponent(ry)
        # the exponent, but where fp32 and fp64 may see amax on two sides of 448 · 2^e
        edge = np.abs(top / (448.0 * np.exp2(ref)) - 1) < 2.0 ** -16
        edge |= np.abs(top / (448.0 * np.exp2(ref - 1.0)) - 1) < 2.0 ** -16
        assert np.all((e == ref) | edge)
        s = np.repeat(np.exp2(e), 32, axis=1)
        v = e4m3_to_f64(codes.cpu().numpy()) * s
        tol = np.maximum(np.abs(ry) * 2.0 ** -4, s * 2.0 ** -10)
        assert np.all(np.abs(v - ry) <= tol * (1 + 2.0 ** -10))


@pytest.mark.gpu
@pytest.mark.parametrize("quant", [None, "e4m3", "mxfp8"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,d,res", [
    (1, 7168, True), (3, 32, False), (70, 128, False), (5, 96, True), (33, 1024, True),
    (700, 2080, True), (2, 16384, False), (2, 33024, True)])
def test_matches_definition(rows, d, res, dtype, quant):
    import sparse_attention_lightning_gb300 as dsa
    g = torch.Generator().manual_seed(rows * 131 + d)
    x = torch.randn(rows, d, generator=g).to(dtype).cuda()
    w = (1 + 0.2 * torch.randn(d, generator=g)).to(dtype).cuda()
    r = torch.randn(rows, d, generator=g).to(dtype).cuda() if res else None
    y, h, codes, scale = dsa.add_rmsnorm(x, w, r, EPS, quant, want_y=True)
    assert y is not None and (h is None) == (r is None)
    _check(x, w, r, EPS, quant, y, h, codes, scale)


@pytest.mark.gpu
@pytest.mark.parametrize("quant", [None, "e4m3"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [1, 7, 31, 129, 1001, 20011])
def test_odd_lengths(d, dtype, quant):
    import sparse_attention_lightning_gb300 as dsa
    g = torch.Generator().manual_seed(d)
    x, r = (torch.randn(9, d, generator=g).to(dtype).cuda() for _ in range(2))
    w = torch.randn(d, generator=g).to(dtype).cuda()
    y, h, codes, scale = dsa.add_rmsnorm(x, w, r, EPS, quant, want_y=True)
    _check(x, w, r, EPS, quant, y, h, codes, scale)


@pytest.mark.gpu
@pytest.mark.parametrize("quant", [None, "e4m3", "mxfp8"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows", [5, 620])
@pytest.mark.parametrize("d", [37, 129, 513, 1025, 2049, 3001, 4096, 4097, 8191, 8192, 8193])
def test_single_elements_and_few_or_many_rows(d, rows, dtype, quant):
    """Rows that start between 16-byte boundaries (a slice of a wider tensor), each way of sharing them out."""
    import sparse_attention_lightning_gb300 as dsa
    if quant == "mxfp8":
        d = d // 32 * 32
    g = torch.Generator().manual_seed(d + rows)
    x, r = (torch.randn(rows, d + 5, generator=g).to(dtype).cuda()[:, 3:3 + d] for _ in range(2))
    w = torch.randn(d, generator=g).to(dtype).cuda()
    y, h, codes, scale = dsa.add_rmsnorm(x, w, r, EPS, quant, want_y=True)
    _check(x, w, r, EPS, quant, y, h, codes, scale)


@pytest.mark.gpu
@pytest.mark.parametrize("quant", [None, "e4m3", "mxfp8"])
@pytest.mark.parametrize("rows", [4, 620])
@pytest.mark.parametrize("d", [32, 160, 256, 288, 512, 1024, 1056])
def test_vectors_and_few_or_many_rows(d, rows, quant):
    import sparse_attention_lightning_gb300 as dsa
    for dtype in (torch.bfloat16, torch.float32):
        g = torch.Generator().manual_seed(d + rows)
        x, r = (torch.randn(rows, d, generator=g).to(dtype).cuda() for _ in range(2))
        w = torch.randn(d, generator=g).to(dtype).cuda()
        y, h, codes, scale = dsa.add_rmsnorm(x, w, r, EPS, quant, want_y=True)
        _check(x, w, r, EPS, quant, y, h, codes, scale)


@pytest.mark.gpu
@pytest.mark.parametrize("off", [0, 8, 3])
def test_strided_slice_and_shapes(off):
    """A slice of a wider projection (aligned and not), leading dimensions, index-key rows."""
    import sparse_attention_lightning_gb300 as dsa
    g = torch.Generator().manual_seed(off)
    wide = torch.randn(6, 11, 200, generator=g).to(torch.bfloat16).cuda()
    x = wide[:, :, off:off + 128]
    w = torch.randn(128, generator=g).to(torch.bfloat16).cuda()
    for quant in ("e4m3", "mxfp8"):
        y, h, codes, scale = dsa.add_rmsnorm(x, w, None, EPS, quant)
        assert y is None and h is None and codes.shape == (6, 11, 128)
        assert scale.shape == ((6, 11) if quant == "e4m3" else (6, 11, 4))
        _check(x.reshape(66, 128), w, None, EPS, quant, None, None, codes.reshape(66, 128),
               scale.reshape(66, -1))
    with pytest.raises(ValueError):
        dsa.add_rmsnorm(wide.transpose(0, 1)[:, :, :128], w)  # rows not evenly spaced
    with pytest.raises(ValueError):
        dsa.add_rmsnorm(wide[:, :, ::2][:, :, :64], w[:64])
    with pytest.raises(ValueError):
        dsa.add_rmsnorm(x, w.float())
    with pytest.raises(ValueError):
        dsa.add_rmsnorm(x, w, quant="int8")
    with pytest.raises(ValueError):
        dsa.add_rmsnorm(x[..., :100], w[:100], quant="mxfp8")


@pytest.mark.gpu
@pytest.mark.parametrize("d", [256, 4096, 40000])
def test_in_place_matches_out_of_place(d):
    import sparse_attention_lightning_gb300 as dsa
    x, r = (torch.randn(37, d, device="cuda").to(torch.bfloat16) for _ in range(2))
    w = torch.randn(d, device="cuda").to(torch.bfloat16)
    y0, h0, _, _ = dsa.add_rmsnorm(x, w, r)
    y1, h1, _, _ = dsa.add_rmsnorm(x, w, r, h=r, y=x)
    assert h1.data_ptr() == r.data_ptr() and torch.equal(y0, x) and torch.equal(h0, r)


@pytest.mark.gpu
@pytest.mark.parametrize("quant", ["e4m3", "mxfp8"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_special_rows(quant, dtype):
    """Zeros, tiny and huge values, NaN and infinity; no row disturbs its neighbours."""
    import sparse_attention_lightning_gb300 as dsa
    x = torch.randn(8, 64, device="cuda").to(dtype)
    w = torch.ones(64, device="cuda", dtype=dtype)
    x[1] = 0
    x[2] = 1e-30                     # eps dominates: y ~ 1e-27
    x[3, 5] = 1e15
    x[4, 7] = float("nan")
    x[5, 9] = float("inf")
    x[6, 32:] = 0                    # an all-zero group
    y, _, codes, scale = dsa.add_rmsnorm(x, w, None, EPS, quant, want_y=True)
    ok = [0, 1, 2, 3, 6, 7]
    _check(x[ok], w, None, EPS, quant, y[ok], None, codes[ok], scale[ok])
    assert torch.isnan(y[4]).all()
    assert torch.isnan(y[5, 9]) and (y[5, :9] == 0).all() and (y[5, 10:] == 0).all()
    c = codes.cpu()
    assert ((c[4] & 0x7F) == 0x7F).all() and (c[5, 9] & 0x7F) == 0x7F
    if quant == "mxfp8":
        s = scale.cpu()
        assert s.max() < 255 and s[1].tolist() == [127, 127] and s[6, 1] == 127
        assert ((c[5, 32:] & 0x7F) == 0).all()  # x · 0 keeps x's sign: codes 0x00 and 0x80
    else:
        assert scale[1] == 1.0


@pytest.mark.gpu
def test_empty_and_graph():
    import sparse_attention_lightning_gb300 as dsa
    w = torch.ones(64, device="cuda", dtype=torch.bfloat16)
    y, _, c, s = dsa.add_rmsnorm(torch.empty(0, 64, device="cuda", dtype=torch.bfloat16), w,
                                 quant="e4m3", want_y=True)
    assert y.shape == (0, 64) and c.numel() == 0 and s.numel() == 0
    x = torch.randn(16, 64, device="cuda").to(torch.bfloat16)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        yg, _, cg, sg = dsa.add_rmsnorm(x, w, quant="e4m3", want_y=True)
    x.copy_(torch.randn(16, 64, device="cuda"))
    graph.replay()
    y, _, c, s = dsa.add_rmsnorm(x, w, quant="e4m3", want_y=True)
    assert torch.equal(y, yg) and torch.equal(c, cg) and torch.equal(s, sg)
