"""The 4-bit latent cache: rows written and read (dsa_write_kv4, dsa_read_kv4) and sparse attention over
it (dsa_sparse_mla_attn4), against the fp64 definitions."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import cache_ops as C
from oracle import kv4_ops as K
from sparse_attention_lightning_gb300 import _abi

BF, F32 = torch.bfloat16, torch.float32
FULL = dict(d_c=512, d_rope=64)


def test_oracle_formats():
    assert K.row_bytes(512, 64) == 416 and K.row_bytes(16, 0) == 16 and K.row_bytes(48, 16) == 64
    assert K.SCALES[1] == 2.0 ** -17 and K.SCALES[8] == 2.0 ** -14 and K.SCALES[0x78] == 1 and K.SCALES[247] == 61440
    for b in range(248):  # a scale byte is the upper part of an fp16 number
        assert np.uint16(b << 7).view(np.float16) == K.SCALES[b]
    x = np.array([[6, -6, 3, 2.5, 3.5, 5, 0.25, 0.75, -0.25, 1.25, 1.75, 0.3, 4.9, 5.1, 0, -1]])
    r = K.decode(K.encode(x, np.zeros((1, 0))), 16, 0)
    assert np.array_equal(r, [[6, -6, 3, 2, 4, 4, 0, 1, 0, 1, 2, 0.5, 4, 6, 0, -1]])
    # of a word's nibbles the low half are even columns
    assert list(K.encode(x, np.zeros((1, 0)))[0][:4]) == [0x57, 0x06 | 0x00, 0x4f, 0x26]


def test_argument_checks():
    L, A = _abi.lib(), 1 << 20
    bad, unsup, wse = _abi.DSA_ERR_INVALID_ARG, _abi.DSA_ERR_UNSUPPORTED, _abi.DSA_ERR_WORKSPACE

    def problem(**kw):
        base = dict(num_seqs=1, total_q=4, total_k=64, max_q_len=4, max_k_len=64, h_idx=4, d_idx=32,
                    h=8, d_c=64, d_rope=16, top_k=8, idx_dtype=0, kv_dtype=0, out_dtype=0,
                    sm_scale=0.0, cu_q=4096, cu_k=8192)
        base.update(kw)
        return _abi.DsaProblem(**base)

    n = ctypes.c_int32(0)
    assert L.dsa_kv4_row_bytes(512, 64, ctypes.byref(n)) == 0 and n.value == 416
    for d_c, d_rope in ((8, 0), (1040, 0), (24, 0), (64, 8), (64, 272)):
        assert L.dsa_kv4_row_bytes(d_c, d_rope, ctypes.byref(n)) == unsup
    assert L.dsa_kv4_row_bytes(512, 64, None) == bad

    def write(p=None, lat=A, ld=64, rope=2 * A, ldr=16, kv4=3 * A, ws=4 * A, wsb=1 << 20):
        return L.dsa_write_kv4(ctypes.byref(p or problem()), lat, ld, rope, ldr, kv4, ws, wsb, None)

    assert write(lat=None) == bad and write(ld=63) == bad and write(rope=None) == bad and write(ldr=15) == bad
    assert write(lat=A + 2) == bad and write(rope=A + 1) == bad and write(kv4=3 * A + 8) == bad and write(kv4=None) == bad
    assert write(kv4=A + 512) == bad and write(kv4=2 * A - 64) == bad      # over the inputs
    assert write(ws=None) == wse and write(wsb=100) == wse
    assert write(problem(d_c=72)) == unsup and write(problem(kv_dtype=2)) == unsup
    assert write(problem(total_q=0, max_q_len=0), lat=None, rope=None) == _abi.DSA_OK

    def read(p=None, kv4=A, out=2 * A, ws=4 * A, wsb=1 << 20):
        return L.dsa_read_kv4(ctypes.byref(p or problem()), kv4, out, ws, wsb, None)

    assert read(kv4=None) == bad and read(out=None) == bad and read(out=2 * A + 4) == bad and read(out=A + 16) == bad
    assert read(ws=None) == wse and read(problem(d_rope=8)) == unsup

    def attn(p=None, q=A, kv4=2 * A, idx=3 * A, out=4 * A, lse=None, ws=5 * A, wsb=1 << 40):
        return L.dsa_sparse_mla_attn4(ctypes.byref(p or problem()), q, kv4, idx, out, lse, ws, wsb, None)

    assert attn(q=None) == bad and attn(kv4=None) == bad and attn(idx=None) == bad and attn(out=None) == bad
    assert attn(lse=A + 4) == bad and attn(q=A + 8) == bad and attn(kv4=A + 8) == bad
    assert attn(ws=None) == wse and attn(wsb=100) == wse
    assert attn(problem(h=129)) == unsup and attn(problem(top_k=2049)) == unsup and attn(problem(kv_dtype=2)) == unsup
    assert attn(problem(total_q=0, max_q_len=0), q=None, idx=None, out=None) == _abi.DSA_OK
    assert attn(problem(max_q_len=0)) == bad


@pytest.mark.parametrize("total_q", [0, 1, 5, 40, 170, 5000])
@pytest.mark.parametrize("h,top_k", [(128, 2048), (16, 999), (1, 1), (64, 130)])
def test_workspace_of_any_device(total_q, h, top_k):
    """Sized without a device too, where a cluster of CTAs has no place."""
    p = _abi.DsaProblem(num_seqs=1, total_q=total_q, total_k=8192, max_q_len=total_q, max_k_len=8192, h_idx=4, d_idx=32, h=h, d_c=512,
                        d_rope=64, top_k=top_k, idx_dtype=0, kv_dtype=_abi.DSA_BF16, out_dtype=_abi.DSA_BF16, sm_scale=0.0,
                        cu_q=4096, cu_k=8192)
    n = ctypes.c_size_t(0)
    assert _abi.lib().dsa_workspace_size(ctypes.byref(p), _abi.OP_SPARSE_MLA_ATTN4, ctypes.byref(n)) == 0 and n.value > 0


class Setup:
    """Sequences with a 4-bit cache, packed or paged; unused bytes of the cache are 0xff (NaN scales, NaN rope columns)."""

    def __init__(self, q_lens, k_lens, h, d_c, d_rope, dtype, top_k=8, page=0, seed=0, spread=1.0, out_dtype=None):
        import sparse_attention_lightning_gb300 as dsa
        g = self.g = torch.Generator().manual_seed(seed)
        D = d_c + d_rope
        self.q_lens, self.k_lens, self.h, self.d_c, self.d_rope, self.page = q_lens, k_lens, h, d_c, d_rope, page
        self.scale, self.top_k, self.dtype = D ** -0.5, top_k, dtype
        self.q = (torch.randn(sum(q_lens), h, D, generator=g) * spread).to(dtype)
        self.rows = [K.encode(torch.randn(n, d_c, generator=g).double().numpy(), torch.randn(n, d_rope, generator=g).numpy())
                     for n in k_lens]
        rb = K.row_bytes(d_c, d_rope)
        kw, self.at = {}, []
        if page:
            need = [-(-n // page) for n in k_lens]
            order = torch.randperm(sum(need) + 2, generator=g).tolist()
            self.host = np.full(((sum(need) + 2) * page, rb), 0xff, np.uint8)
            table = torch.full((len(k_lens), max(max(need), 1)), -1, dtype=torch.int32)
            for b, n in enumerate(k_lens):
                pages = [order.pop() for _ in range(need[b])]
                table[b, :len(pages)] = torch.tensor(pages, dtype=torch.int32)
                self.at.append(np.array([pages[s // page] * page + s % page for s in range(n)], dtype=int))
            kw = dict(block_table=table.cuda(), page_size=page, num_pages=sum(need) + 2)
        else:
            self.host = np.full((sum(k_lens), rb), 0xff, np.uint8)
            for c, n in zip(np.cumsum([0] + k_lens), k_lens):
                self.at.append(np.arange(c, c + n))
        for at, rows in zip(self.at, self.rows):
            self.host[at] = rows
        self.kv4 = torch.from_numpy(self.host).cuda()
        cu = lambda v: torch.tensor([0] + list(np.cumsum(v)), dtype=torch.int32).cuda()  # noqa: E731
        name = {BF: "bf16", F32: "f32"}
        self.prob = dsa.Problem(cu(q_lens), cu(k_lens), q_lens=q_lens, k_lens=k_lens, h_idx=4, d_idx=32, h=h, d_c=d_c,
                                d_rope=d_rope, top_k=top_k, idx_dtype="f32", kv_dtype=name[dtype],
                                out_dtype=name[out_dtype or dtype], **kw)

    def tokens(self):
        """(query row, sequence, position)."""
        t = 0
        for b, (T, L) in enumerate(zip(self.q_lens, self.k_lens)):
            for i in range(T):
                yield t, b, L - T + i
                t += 1

    def draw_idx(self, holes=0.0):
        """Distinct positions in no order, -1 behind them and, with holes, among them."""
        idx = torch.full((sum(self.q_lens), self.top_k), -1, dtype=torch.int32)
        for t, _, pos in self.tokens():
            n = min(self.top_k, pos + 1)
            idx[t, :n] = torch.randperm(pos + 1, generator=self.g)[:n].to(torch.int32)
            if holes:
                idx[t, torch.rand(self.top_k, generator=self.g) < holes] = -1
        return idx

    def attend(self, idx, **kw):
        import sparse_attention_lightning_gb300 as dsa
        return dsa.sparse_mla_attn4(self.prob, self.q.cuda(), self.kv4, idx.cuda(), **kw)

    def check(self, out, lse, idx, rows=None):
        """Errors counted, per element.  Decoded keys are exact.  A logit is off by at most δ = (D + 2) · 2^-24 · max_x
        scale · Σ_c |q_c k_c| (fp32 accumulation in any order, then the scale), which changes every p by a factor within
        e^(2δ) and lse by δ.  bf16 on the tensor cores: each p is rounded to bf16 (2^-8), the output too (2^-8 of it).  fp32
        sums over n entries: below 2^-24 · n of Σ p|v|; 2^-20 for 2^x, the logarithm and the merge of pieces."""
        out, lse = out.float().cpu().double().numpy(), lse.cpu().double().numpy()
        D = self.d_c + self.d_rope
        decoded = {}
        for t, b, pos in self.tokens():
            if rows is not None and t not in rows:
                continue
            if b not in decoded:
                decoded[b] = K.decode(self.host[self.at[b]], self.d_c, self.d_rope)
            i = idx[t].numpy()
            keys = decoded[b][i[(i >= 0) & (i <= pos)]]
            ro, rl, mag, top = C.attend(self.q[t].double().numpy(), keys, self.d_c, self.scale)
            delta = (D + 2) * 2.0 ** -24 * top
            rel = 2 * delta + len(keys) * 2.0 ** -24 + 2.0 ** -20
            half = 2.0 ** -8 if self.dtype == BF else 0.0
            rounding = 2.0 ** -8 if self.prob.out_dtype == _abi.DSA_BF16 else 2.0 ** -24
            tol = (rel[:, None] + half) * mag * (1 + rounding) + rounding * np.abs(ro) + 1e-38
            err = np.abs(out[t] - ro)
            assert np.all(err <= tol), (t, (err / tol).max())
            if len(keys) == 0:
                assert np.all(np.isneginf(lse[t])) and np.all(out[t] == 0)
                continue
            bound = delta + (len(keys) + 8) * 2.0 ** -24 + 2.0 ** -20 * (1 + np.abs(rl))
            assert np.all(np.abs(lse[t] - rl) <= bound), (t, np.abs(lse[t] - rl).max())


# ---------------------------------------------------------------------------
# Rows.

ROWS = [([1], [1], 512, 64, 0), ([1, 3, 0, 2], [1, 3, 7, 40], 512, 64, 16), ([5, 1], [70, 64], 64, 16, 64),
        ([9], [33], 16, 0, 0), ([4, 4], [4, 20], 48, 16, 32), ([2, 1, 1], [300, 1, 2], 1024, 256, 128),
        ([130], [200], 512, 0, 0), ([1] * 70, list(range(1, 71)), 128, 64, 16)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("q_lens,k_lens,d_c,d_rope,page", ROWS)
@pytest.mark.parametrize("aligned", [True, False])
def test_rows_written_and_read(q_lens, k_lens, d_c, d_rope, page, dtype, aligned):
    """Bytes equal to the definition's, other rows as they were, and the values back."""
    import sparse_attention_lightning_gb300 as dsa
    s = Setup(q_lens, k_lens, 2, d_c, d_rope, dtype, page=page, seed=d_c)
    wide = torch.randn(sum(q_lens), d_c + d_rope + (8 if aligned else 5), generator=s.g)
    wide = (wide * torch.exp(torch.randn(wide.shape[0], 1, generator=s.g) * 4)).to(dtype)
    lat, rope = wide[:, :d_c], wide[:, d_c:d_c + d_rope]
    dev = wide.cuda()
    ws = dsa.Workspace()
    got = dsa.write_kv4(s.prob, dev[:, :d_c], dev[:, d_c:d_c + d_rope] if d_rope else None, s.kv4, ws=ws)
    assert got is s.kv4 and ws.status() == 0
    new = K.encode(lat.double().numpy(), rope.double().numpy())
    for t, b, pos in s.tokens():
        s.host[s.at[b][pos]] = new[t]
    assert np.array_equal(s.kv4.cpu().numpy(), s.host)
    out = dsa.read_kv4(s.prob, s.kv4, ws=ws)
    want = np.concatenate([K.decode(s.host[at], d_c, d_rope) for at in s.at])
    assert out.dtype == dtype and np.array_equal(out.double().cpu().numpy(), want) and ws.status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
def test_every_rounding(dtype):
    """Groups whose largest value walks through scales and their ties, elements through codes and theirs."""
    import sparse_attention_lightning_gb300 as dsa
    n, d_c = 2048, 512
    g = torch.Generator().manual_seed(1)
    amax = torch.exp2(torch.rand(n, d_c // 16, generator=g) * 40 - 22)            # from 0 to beyond the largest scale
    amax[:600] = 6 * torch.exp2(torch.randint(-18, 17, (600, 32), generator=g).float()) \
        * (1 + torch.randint(0, 17, (600, 32), generator=g).float() / 16)        # scales and the middles between them
    part = torch.rand(n, d_c // 16, 16, generator=g)
    part[:1200] = torch.randint(0, 49, (1200, 32, 16), generator=g).float() / 48  # codes and the middles between them
    part[:, :, 3] = 1
    sign = torch.randint(0, 2, part.shape, generator=g) * 2 - 1
    x = (amax[:, :, None] * part * sign).reshape(n, d_c)
    x[7], x[8, :16], x[9, 16:32] = 0, -0.0, 3e38
    x[10, 5], x[11, 40], x[12, 100] = float("nan"), float("inf"), -float("inf")
    x[13, :16] = 1e-38
    if dtype == F32:  # next to the ties
        up = torch.randint(-1, 2, x.shape, generator=g).to(torch.int32)
        near = (x.view(torch.int32) + up).view(torch.float32)
        x[20:1000] = torch.where(x[20:1000] != 0, near[20:1000], x[20:1000])
    x = x.to(dtype)
    s = Setup([n], [n], 1, d_c, 16, dtype, seed=2)
    rope = torch.randn(n, 16, generator=g)
    rope[0, 0], rope[1, 1], rope[2, 2], rope[3, 3] = float("inf"), -float("inf"), float("nan"), 3.4e38
    rope = rope.to(dtype)
    dsa.write_kv4(s.prob, x.cuda(), rope.cuda(), s.kv4)
    with np.errstate(over="ignore"):
        want = K.encode(x.double().numpy(), rope.double().numpy())
    got = s.kv4.cpu().numpy()
    at = d_c // 2
    nan = got[2, at + 4:at + 6].view("<u2") & 0x7fff
    assert nan[0] > 0x7f80                                       # any NaN
    got[2, at + 4:at + 6] = want[2, at + 4:at + 6]
    assert np.array_equal(got, want)
    out = dsa.read_kv4(s.prob, s.kv4).double().cpu().numpy()
    assert np.array_equal(out, K.decode(want, d_c, 16), equal_nan=True)
    assert np.isnan(out[10, :16]).all() and not np.isnan(out[10, 16:d_c]).any()


@pytest.mark.gpu
def test_every_byte_decodes():
    """Every scale byte with every code."""
    import sparse_attention_lightning_gb300 as dsa
    s = Setup([1], [256], 1, 512, 16, F32)
    rows = np.zeros((256, K.row_bytes(512, 16)), np.uint8)
    rows[:, :256] = np.random.default_rng(0).integers(0, 256, (256, 256))
    rows[:, 288:320] = np.arange(256)[:, None]
    rows[:, 256:288] = np.random.default_rng(1).integers(0, 0x7f, (256, 32))
    for dtype in ("f32", "bf16"):
        P = s.prob if dtype == "f32" else Setup([1], [256], 1, 512, 16, BF).prob
        out = dsa.read_kv4(P, torch.from_numpy(rows).cuda()).double().cpu().numpy()
        assert np.array_equal(out, K.decode(rows, 512, 16), equal_nan=True)


@pytest.mark.gpu
def test_bad_pages_and_sequences_leave_rows():
    import sparse_attention_lightning_gb300 as dsa
    s = Setup([2, 1, 1], [20, 40, 30], 2, 64, 16, BF, page=16, seed=3)
    lat, rope = torch.randn(4, 64).bfloat16().cuda(), torch.randn(4, 16).bfloat16().cuda()
    ws = dsa.Workspace()
    for page in (-1, 99):
        table = s.prob.block_table
        keep = int(table[1, 2])
        table[1, 2] = page                                       # positions 32 .. 39 of sequence 1
        before = s.kv4.clone()
        dsa.write_kv4(s.prob, lat, rope, s.kv4, ws=ws)
        assert ws.status() == _abi.DSA_FLAG_BAD_SEQS
        ws.clear_status()
        changed = (s.kv4 != before).any(dim=1).nonzero()[:, 0].tolist()
        assert changed == sorted(int(s.at[b][p]) for b, p in ((0, 18), (0, 19), (2, 29)))
        out = torch.full((90, 80), 7.0, dtype=BF, device="cuda")
        dsa.read_kv4(s.prob, s.kv4, out=out, ws=ws)
        assert ws.status() == _abi.DSA_FLAG_BAD_INDEX
        ws.clear_status()
        assert (out[52:60] == 7).all() and not (out[:52] == 7).all(dim=1).any() and not (out[60:] == 7).all(dim=1).any()
        table[1, 2] = keep
        s.kv4.copy_(before)
    s.prob.cu_q.copy_(torch.tensor([0, 1, 4, 4], dtype=torch.int32))   # T_1 = 3, max_q_len = 2
    before = s.kv4.clone()
    dsa.write_kv4(s.prob, lat, rope, s.kv4, ws=ws)
    assert ws.status() == _abi.DSA_FLAG_BAD_SEQS
    assert (s.kv4 != before).any(dim=1).nonzero()[:, 0].tolist() == [int(s.at[0][19])]


# ---------------------------------------------------------------------------
# Attention.

ATTN = [
    # q_lens, k_lens, heads, d_c, d_rope, top_k, page
    ([1], [1], 1, 512, 64, 1, 0), ([1], [1], 128, 512, 64, 2048, 0), ([1, 1, 1], [40, 64, 65], 128, 512, 64, 64, 0),
    ([1] * 5, [3000, 17, 2048, 129, 1], 128, 512, 64, 2048, 64), ([3, 1, 0, 2], [300, 200, 50, 2], 16, 512, 64, 130, 16),
    ([1, 4], [513, 700], 20, 512, 64, 500, 256), ([30], [30], 64, 512, 64, 33, 0), ([2], [5000], 127, 512, 64, 1999, 128),
    ([1] * 33, [100 + 60 * i for i in range(33)], 8, 512, 64, 257, 64),
    ([2, 1], [100, 30], 8, 64, 16, 32, 16), ([5], [90], 20, 256, 32, 70, 0), ([1, 1], [80, 20], 3, 16, 0, 9, 0),
    ([1, 2], [50, 60], 17, 1024, 256, 40, 32), ([2], [33], 4, 512, 0, 16, 0), ([1], [200], 5, 128, 64, 100, 64),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,out_dtype", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)])
@pytest.mark.parametrize("q_lens,k_lens,h,d_c,d_rope,top_k,page", ATTN)
def test_attention(q_lens, k_lens, h, d_c, d_rope, top_k, page, dtype, out_dtype):
    import sparse_attention_lightning_gb300 as dsa
    s = Setup(q_lens, k_lens, h, d_c, d_rope, dtype, top_k, page, seed=h + top_k, spread=2.0, out_dtype=out_dtype)
    idx = s.draw_idx()
    ws = dsa.Workspace()
    out, lse = s.attend(idx, ws=ws)
    assert ws.status() == 0
    s.check(out, lse, idx)
    again, lse2 = s.attend(idx, want_lse=False)
    assert torch.equal(out, again) and lse2 is None


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,h,d_c,d_rope", [(BF, 128, 512, 64), (BF, 16, 512, 64), (F32, 8, 64, 16), (BF, 8, 256, 32)])
@pytest.mark.parametrize("page", [0, 64])
def test_skipped_entries(dtype, h, d_c, d_rope, page):
    """Holes, whole steps of padding, rows without an entry, repeated entries, positions ahead of the query, pages outside."""
    import sparse_attention_lightning_gb300 as dsa
    s = Setup([4, 1, 1], [900, 400, 300], h, d_c, d_rope, dtype, 400, page, seed=5)
    idx = s.draw_idx(holes=0.4)
    idx[0] = -1
    idx[1, :320] = -1
    idx[2, 100:] = -1
    idx[3, 7:200] = 5
    ws = dsa.Workspace()
    out, lse = s.attend(idx, ws=ws)
    assert ws.status() == 0
    s.check(out, lse, idx)
    idx[4, 3], idx[4, 90], idx[5, 0] = 400, -2, 1 << 30
    out, lse = s.attend(idx, ws=ws)
    assert ws.status() == _abi.DSA_FLAG_BAD_INDEX
    s.check(out, lse, idx)
    if page:
        ws.clear_status()
        s.prob.block_table[1, 2], s.prob.block_table[1, 3] = -1, s.prob.num_pages
        out, lse = s.attend(idx, ws=ws)
        assert ws.status() == _abi.DSA_FLAG_BAD_INDEX
        lost = idx.clone()
        lost[4, (idx[4] >= 128) & (idx[4] < 256)] = -1
        s.check(out, lse, lost)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,h,d_c,d_rope", [(BF, 128, 512, 64), (BF, 16, 512, 64), (F32, 8, 64, 16)])
def test_values_that_are_not_finite(dtype, h, d_c, d_rope):
    """A selected key with a NaN makes every output of the query's heads NaN, one that is not selected nothing; logits of
    +inf and -inf as the formula has them."""
    s = Setup([1] * 4, [200] * 4, h, d_c, d_rope, dtype, 150, seed=6)
    idx = s.draw_idx()
    at, rope = d_c // 2 + 2 * d_rope, d_c // 2
    sel = [idx[t].tolist() for t in range(4)]
    free = [next(p for p in range(200) if p not in sel[t]) for t in range(4)]
    for t in range(4):
        s.host[s.at[t][free[t]]] = 0xff                                     # not selected: NaN everywhere
    s.host[s.at[1][sel[1][70]], at + 1] = 0xff                              # 16 NaN columns
    inf = np.array([0x7f80], "<u2").view(np.uint8)
    s.host[s.at[2][sel[2][3]], rope:rope + 2] = inf                         # a rope column of +inf
    s.host[s.at[3][sel[3][149]], rope:rope + 2] = inf
    s.q[2, :, d_c] = s.q[2, :, d_c].abs() + 1                               # logit +inf: NaN outputs
    s.q[3, :, d_c] = -s.q[3, :, d_c].abs() - 1                              # logit -inf: weight 0
    s.kv4 = torch.from_numpy(s.host).cuda()
    out, lse = s.attend(idx)
    assert torch.isnan(out[1]).all() and torch.isnan(lse[1]).all()
    assert torch.isnan(out[2]).all()
    idx[3, 149] = -1
    s.check(out, lse, idx, rows={0, 3})
    # all logits -inf
    lone = torch.full_like(idx, -1)
    lone[3, 0] = sel[3][149]
    out, lse = s.attend(lone)
    assert (out[3] == 0).all() and torch.isneginf(lse[3]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("h", [128, 16])
def test_extreme_scales_and_logits(h):
    """Scales at both ends of their range, logits of several thousands that grow along the row."""
    s = Setup([1, 1, 1], [700, 700, 700], h, 512, 64, BF, 640, seed=7)
    s.host[s.at[0], 384:416] = 247
    s.host[s.at[1], 384:416] = 1
    q = s.q.float()
    q[0] *= 2.0 ** -18
    s.q = q.bfloat16()
    rows = s.host[s.at[2]]
    rows[:, 384:416] = (0x58 + np.arange(700) // 20)[:, None].astype(np.uint8)  # to 2^-4 .. 2^0
    s.host[s.at[2]] = rows
    s.q[2] *= 8
    s.kv4 = torch.from_numpy(s.host).cuda()
    idx = s.draw_idx().sort(dim=1).values
    s.check(*s.attend(idx), idx)


@pytest.mark.gpu
@pytest.mark.parametrize("h,top_k", [(128, 70), (40, 200), (16, 513)])
def test_more_queries_than_sms(h, top_k):
    """Several queries a CTA one after another: full rows, short ones, rows without an entry, in every order."""
    s = Setup([300, 1, 90], [300, 40, 700], h, dtype=BF, top_k=top_k, page=64, seed=h, spread=2.0, **FULL)
    idx = s.draw_idx()
    g = torch.Generator().manual_seed(1)
    idx[torch.rand(idx.shape[0], generator=g) < 0.3] = -1
    idx[5:340:7, 3:] = -1
    out, lse = s.attend(idx)
    s.check(out, lse, idx, rows=set(range(0, 391, 3)) | {390})
    for _ in range(3):
        again, lse2 = s.attend(idx)
        assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.gpu
@pytest.mark.parametrize("queries,h,top_k,out_dtype", [
    (1, 128, 2048, BF), (2, 40, 2000, F32), (5, 16, 2048, BF), (9, 64, 1999, F32), (14, 128, 2048, F32), (30, 128, 2048, BF),
    (30, 65, 777, F32), (33, 20, 2048, BF), (60, 128, 2048, BF), (61, 96, 1030, F32), (76, 33, 130, BF), (170, 128, 2048, BF),
    (180, 16, 2048, F32)])
def test_pieces_of_a_query(queries, h, top_k, out_dtype):
    """Queries cut into pieces, joined by the CTAs of a cluster or by a merge, in one round and in several: pieces without an
    entry, queries without any, one entry behind nothing; the same again from a captured graph."""
    import sparse_attention_lightning_gb300 as dsa
    s = Setup([queries], [2100 + queries], h, dtype=BF, top_k=top_k, page=64, seed=queries, spread=2.0, out_dtype=out_dtype, **FULL)
    idx = s.draw_idx()
    if queries > 4:
        idx[1, :top_k * 3 // 4] = -1
        idx[2, top_k // 5:] = -1
        idx[3] = -1
        idx[4, :-1] = -1
        idx[queries - 1, top_k // 3:top_k * 2 // 3] = -1
    ws = dsa.Workspace()
    out, lse = s.attend(idx, ws=ws)
    assert ws.status() == 0
    s.check(out, lse, idx, rows=set(range(0, queries, 1 + queries // 12)) | {0, 1, 2, 3, 4, queries - 1})
    q, dev, out2, lse2 = s.q.cuda(), idx.cuda(), torch.zeros_like(out), torch.zeros_like(lse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dsa.sparse_mla_attn4(s.prob, q, s.kv4, dev, out=out2, lse=lse2, ws=ws)
    for _ in range(3):
        out2.fill_(3), lse2.fill_(3)
        g.replay()
        assert torch.equal(out, out2) and torch.equal(lse, lse2)


@pytest.mark.gpu
@pytest.mark.parametrize("h", [128, 16])
def test_queries_of_any_magnitude(h):
    """Heads of zeros, of subnormal and of huge numbers, of widely spread ones, latent and rope columns apart; infinities and NaNs
    stay in their head."""
    s = Setup([1], [150], h, dtype=BF, top_k=130, seed=12, **FULL)
    q = s.q.float()[0]
    wide = torch.exp2(torch.rand(h, 576, generator=s.g) * 60 - 50)
    q[1] = 0
    q[2] *= 2.0 ** -130
    q[3] *= 2.0 ** 14
    q[4] *= wide[4]
    q[5, :512], q[5, 512:] = q[5, :512] * 2.0 ** -60, q[5, 512:]
    q[6, :512], q[6, 512:] = q[6, :512], q[6, 512:] * 2.0 ** -60
    q[7, :512], q[7, 512:] = 0, q[7, 512:] * 2.0
    q[8, 7:] = 0
    odd = {9: ("nan", 3), 10: ("inf", 100), 11: ("-inf", 511), 12: ("nan", 540), 13: ("inf", 575)}
    for head, (v, c) in odd.items():
        q[head, c] = float(v)
    s.q = q.bfloat16()[None]
    idx = s.draw_idx()
    out, lse = s.attend(idx)
    keys = K.decode(s.host[s.at[0]], 512, 64)[idx[0].numpy()]
    for head, (v, c) in odd.items():
        nan = v == "nan" or (keys[:, c] * (1 if v == "inf" else -1) > 0).any() or (keys[:, c] == 0).any()
        assert bool(torch.isnan(out[0, head]).all()) == bool(nan), head
    rest = [i for i in range(h) if i not in odd]
    q64 = s.q[0].double().numpy()[rest]
    ro, rl, mag, top = C.attend(q64, keys, 512, s.scale)
    delta = 578 * 2.0 ** -24 * top
    rel = 2 * delta + 130 * 2.0 ** -24 + 2.0 ** -20
    err = np.abs(out[0].float().cpu().double().numpy()[rest] - ro)
    assert np.all(err <= (rel[:, None] + 2.0 ** -8) * mag * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ro) + 1e-38)
    assert np.all(np.abs(lse[0].cpu().double().numpy()[rest] - rl) <= delta + 138 * 2.0 ** -24 + 2.0 ** -20 * (1 + np.abs(rl)))


@pytest.mark.gpu
def test_no_queries():
    import sparse_attention_lightning_gb300 as dsa
    s = Setup([0, 0], [30, 5], 128, dtype=BF, top_k=16, seed=3, **FULL)
    out, lse = s.attend(torch.empty(0, 16, dtype=torch.int32))
    assert out.shape == (0, 128, 512) and lse.shape == (0, 128)
    before = s.kv4.clone()
    none = torch.empty(0, 576).bfloat16().cuda()
    dsa.write_kv4(s.prob, none[:, :512], none[:, 512:], s.kv4)
    assert torch.equal(s.kv4, before) and dsa.read_kv4(s.prob, s.kv4).shape == (35, 576)


@pytest.mark.gpu
def test_checked_build_raises_no_flag_and_matches():
    import sparse_attention_lightning_gb300 as dsa
    from sparse_attention_lightning_gb300 import build
    build.build(checked=True)
    for h, dims, dtype in ((128, FULL, BF), (16, FULL, BF), (4, dict(d_c=64, d_rope=16), F32)):
        s = Setup([3, 1, 30], [700, 2500, 90], h, dtype=dtype, top_k=333, page=64, seed=h, **dims)
        idx = s.draw_idx(holes=0.2)
        want = s.attend(idx)
        with _abi.using(_abi.CHECKED_LIB_PATH):
            ws = dsa.Workspace()
            got = s.attend(idx, ws=ws)
            assert ws.status() == 0
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.gpu
def test_bad_sequences_are_reported():
    import sparse_attention_lightning_gb300 as dsa
    for h, dtype, dims in ((128, BF, FULL), (4, F32, dict(d_c=64, d_rope=16))):
        s = Setup([2, 2], [130, 130], h, dtype=dtype, top_k=70, seed=8, **dims)
        idx = s.draw_idx()
        out0, lse0 = s.attend(idx)
        ws = dsa.Workspace()
        out, lse = torch.full_like(out0, 7.0), torch.full_like(lse0, 7.0)
        s.prob.cu_q.copy_(torch.tensor([0, 1, 4], dtype=torch.int32))  # T_1 = 3, max_q_len = 2
        s.attend(idx, out=out, lse=lse, ws=ws)
        assert ws.status() & _abi.DSA_FLAG_BAD_SEQS and (out[1:] == 7.0).all() and (lse[1:] == 7.0).all()


@pytest.mark.gpu
def test_streams_graphs_and_refusals():
    import sparse_attention_lightning_gb300 as dsa
    s = Setup([1, 1], [3000, 2500], 128, 512, 64, BF, 2048, page=64, seed=9)
    idx = s.draw_idx().cuda()
    q, lat, rope = s.q.cuda(), torch.randn(2, 512).bfloat16().cuda(), torch.randn(2, 64).bfloat16().cuda()
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    P = s.prob

    def step(ws=None):
        dsa.write_kv4(P, lat, rope, s.kv4, ws=ws)
        return (*dsa.sparse_mla_attn4(P, q, s.kv4, idx, ws=ws), dsa.read_kv4(P, s.kv4, ws=ws))

    want = step()
    torch.cuda.synchronize()
    graphs = []
    with pytest.raises(ValueError, match="of its own"):
        with torch.cuda.graph(torch.cuda.CUDAGraph(), stream=side[0]):
            dsa.sparse_mla_attn4(P, q, s.kv4, idx)
    torch.cuda.synchronize()
    for st in side:  # two graphs, each with its workspace, replayed at once
        g, ws = torch.cuda.CUDAGraph(), dsa.Workspace(nbytes=P.workspace_size(_abi.OP_SPARSE_MLA_ATTN4))
        with torch.cuda.graph(g, stream=st):
            got = step(ws)
        graphs.append((g, got, ws))
    for _ in range(20):
        for st, (g, _, _) in zip(side, graphs):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for _, got, ws in graphs:
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and ws.status() == 0
    for bad in (lambda: dsa.write_kv4(P, lat[:1], rope, s.kv4), lambda: dsa.write_kv4(P, lat.float(), rope, s.kv4),
                lambda: dsa.write_kv4(P, lat, None, s.kv4), lambda: dsa.write_kv4(P, lat, rope, s.kv4[:, :400]),
                lambda: dsa.write_kv4(P, lat, rope, s.kv4[1:]), lambda: dsa.write_kv4(P, lat.cpu(), rope, s.kv4),
                lambda: dsa.write_kv4(P, lat.t().contiguous().t(), rope, s.kv4),
                lambda: dsa.read_kv4(P, s.kv4.view(torch.int8)), lambda: dsa.read_kv4(P, s.kv4.cpu()),
                lambda: dsa.read_kv4(P, s.kv4, out=torch.empty(5500, 576).cuda()),
                lambda: dsa.sparse_mla_attn4(P, q.float(), s.kv4, idx), lambda: dsa.sparse_mla_attn4(P, q, s.kv4, idx.long()),
                lambda: dsa.sparse_mla_attn4(P, q, s.kv4[:-64], idx), lambda: dsa.sparse_mla_attn4(P, q, s.kv4, idx[:, :9]),
                lambda: dsa.sparse_mla_attn4(P, q, s.kv4, idx, out=torch.empty(2, 128, 512).cuda())):
        with pytest.raises(ValueError):
            bad()


# ---------------------------------------------------------------------------
# Together.

@pytest.mark.gpu
def test_a_decode_loop_over_a_forked_cache():
    """A prompt is rotated, written, forked into samples that each write their own tokens; pages are freed and compacted on
    the way; attention and the rows read back are those of each sample's own history."""
    import sparse_attention_lightning_gb300 as dsa
    d_c, d_rope, h, page, width, pool = 512, 64, 16, 16, 8, 40
    g = torch.Generator().manual_seed(10)
    rot = dsa.Rotary(d_rope, sections=[16, 8, 8])
    freq, axis = [10000.0 ** (-i / 32) for i in range(32)], [0] * 16 + [1] * 8 + [2] * 8
    i32 = lambda v: torch.tensor(v, dtype=torch.int32).cuda()  # noqa: E731
    table, refs = torch.full((5, width), -1, dtype=torch.int32).cuda(), torch.zeros(pool, dtype=torch.int32).cuda()
    kv4 = torch.full((pool * page, 416), 0xff, dtype=torch.uint8).cuda()
    ws = dsa.Workspace()
    lens, history = [0] * 5, [np.zeros((0, 416), np.uint8) for _ in range(5)]

    def append(rows, n):
        """n tokens for each of the rows: attention over all positions, in random order."""
        new = [lens[r] + n for r in rows]
        held = dsa.reserve_pages(table, refs, i32(rows), i32([lens[r] for r in rows]), i32(new), page, caches=[kv4], ws=ws)
        assert held.cpu().tolist() == new
        B, T = len(rows), n * len(rows)
        cu = lambda v: i32([0] + list(np.cumsum(v)))  # noqa: E731
        P = dsa.Problem(cu([n] * B), cu(new), q_lens=[n] * B, k_lens=new, h_idx=4, d_idx=32, h=h, d_c=d_c, d_rope=d_rope,
                        top_k=100, idx_dtype="f32", kv_dtype="bf16", block_table=table[i32(rows).long()], page_size=page,
                        num_pages=pool)
        lat, rope = torch.randn(T, d_c, generator=g).bfloat16(), torch.randn(T, d_rope, generator=g).bfloat16()
        q = torch.randn(T, h, d_c + d_rope, generator=g).bfloat16()
        pos = torch.tensor([[lens[r] + i for r in rows for i in range(n)], [i * 7 % 50 for i in range(T)], [3] * T],
                           dtype=torch.int32)
        qd = q.cuda()
        dsa.rotate_axes(qd[..., d_c:], pos.cuda(), rot, out=qd[..., d_c:])
        k = dsa.rotate_axes(rope.cuda(), pos.cuda(), rot)
        dsa.write_kv4(P, lat.cuda(), k, kv4, ws=ws)
        angle = pos.double().numpy()[axis].T * np.array(freq)
        assert np.abs(k.double().cpu().numpy() - K.rotate(rope.double().numpy(), angle, True)).max() < 0.05
        rows4 = K.encode(lat.double().numpy(), k.double().cpu().numpy())
        for j, r in enumerate(rows):
            history[r] = np.concatenate([history[r], rows4[j * n:(j + 1) * n]])
            lens[r] = new[j]
        idx = torch.full((T, 100), -1, dtype=torch.int32)
        for j, r in enumerate(rows):
            for i in range(n):
                m = min(100, lens[r] - n + i + 1)
                idx[j * n + i, :m] = torch.randperm(lens[r] - n + i + 1, generator=g)[:m].to(torch.int32)
        out, lse = dsa.sparse_mla_attn4(P, qd, kv4, idx.cuda(), ws=ws)
        check = Setup.__new__(Setup)
        check.__dict__.update(q_lens=[n] * B, k_lens=new, d_c=d_c, d_rope=d_rope, prob=P, dtype=BF, scale=576 ** -0.5,
                              q=qd.cpu(), host=np.concatenate([history[r] for r in rows]),
                              at=[np.arange(e - m, e) for e, m in zip(np.cumsum(new), new)])
        check.check(out, lse, idx)
        back = dsa.read_kv4(P, kv4, ws=ws).double().cpu().numpy()
        assert np.array_equal(back, K.decode(check.host, d_c, d_rope))
        return P, qd, lse

    append([0], 37)
    P, qd, lse0 = append([0], 1)
    full = dsa.read_kv4(P, kv4, ws=ws)  # dense attention over the decoded rows agrees
    packed = dsa.Problem(P.cu_q, P.cu_k, q_lens=P.q_lens, k_lens=P.k_lens, h_idx=4, d_idx=32, h=h, d_c=d_c, d_rope=d_rope,
                         top_k=100, idx_dtype="f32", kv_dtype="bf16")
    _, lse = dsa.prefix_mla_attn(packed, qd, full, ws=ws)
    assert (lse - lse0).abs().max() < 1e-4
    for r in (1, 2, 3, 4):
        lens[r], history[r] = lens[0], history[0].copy()
    dsa.fork_pages(table, refs, i32([0] * 4), i32([1, 2, 3, 4]), i32([lens[0]] * 4), page, ws=ws)
    append([1, 2, 3, 4], 2)
    append([0, 2], 11)
    dsa.free_pages(table, refs, i32([0, 3]), ws=ws)
    lens[0], history[0] = 0, history[0][:0]
    lens[3], history[3] = 0, history[3][:0]
    before = int((refs > 0).sum())
    _, live = dsa.compact_pages(table, refs, page, caches=[kv4], ws=ws)
    assert int(live) == before and int((refs[:before] > 0).sum()) == before
    append([1, 2, 4], 9)
    dsa.fork_pages(table, refs, i32([2]), i32([3]), i32([20]), page, ws=ws)
    lens[3], history[3] = 20, history[2][:20]
    append([3, 1], 3)
    assert ws.status() == 0
