"""Dense MLA attention over a shared prefix (dsa_prefix_mla_attn) against the fp64 definition."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import cache_ops as C
from sparse_attention_lightning_gb300 import _abi

BF, F32 = torch.bfloat16, torch.float32


def test_oracle_is_softmax_attention():
    rng = np.random.default_rng(0)
    q, k = rng.normal(size=(3, 8)), rng.normal(size=(5, 8))
    out, lse, _, _ = C.attend(q, k, 6, 0.5)
    ref = torch.nn.functional.scaled_dot_product_attention(
        torch.from_numpy(q)[None], torch.from_numpy(k)[None], torch.from_numpy(k[:, :6])[None], scale=0.5)
    assert np.allclose(out, ref[0].numpy()) and np.allclose(np.exp(lse), np.exp(q @ k.T / 2).sum(1))


def _problem(**kw):
    base = dict(num_seqs=1, total_q=4, total_k=64, max_q_len=4, max_k_len=64, h_idx=4, d_idx=32,
                h=8, d_c=64, d_rope=16, top_k=8, idx_dtype=0, kv_dtype=0, out_dtype=0,
                sm_scale=0.0, cu_q=4096, cu_k=8192)
    base.update(kw)
    return _abi.DsaProblem(**base)


def test_argument_checks():
    L, A = _abi.lib(), 1 << 20
    bad, unsup = _abi.DSA_ERR_INVALID_ARG, _abi.DSA_ERR_UNSUPPORTED

    def call(p=None, n=10, pre=A, table=None, q=A, kv=A, out=A, lse=None, ws=A, wsb=1 << 40):
        return L.dsa_prefix_mla_attn(ctypes.byref(p or _problem()), n, pre, table, q, kv, out, lse,
                                     ws, wsb, None)

    assert call(n=-1) == bad and call(n=(1 << 30) - 64) == unsup
    assert call(pre=None) == bad                                # a prefix without rows
    assert call(table=A) == bad                                 # both kinds of rows
    assert call(pre=None, table=A) == bad                       # a table without pages
    paged = _problem(page_size=32, max_pages=2, num_pages=3, block_table=1 << 16)
    assert call(paged, pre=None, table=A + 2) == bad
    assert call(pre=A + 8) == bad and call(q=None) == bad and call(kv=None) == bad
    assert call(out=None) == bad and call(lse=A + 4) == bad
    assert call(ws=None) == _abi.DSA_ERR_WORKSPACE and call(wsb=100) == _abi.DSA_ERR_WORKSPACE
    assert call(_problem(h=129)) == unsup and call(_problem(kv_dtype=2)) == unsup
    assert call(_problem(total_q=0, max_q_len=0), q=None, out=None) == _abi.DSA_OK  # no rows: nothing to do


class Setup:
    """A seeded problem: packed or paged caches whose unused rows hold NaN."""

    def __init__(self, q_lens, k_lens, h, d_c, d_rope, P, dtype, page=0, seed=0, spread=1.0):
        import sparse_attention_lightning_gb300 as dsa
        g = torch.Generator().manual_seed(seed)
        D = d_c + d_rope
        self.q_lens, self.k_lens, self.h, self.d_c, self.P, self.page = q_lens, k_lens, h, d_c, P, page
        self.scale = D ** -0.5
        self.q = (torch.randn(sum(q_lens), h, D, generator=g) * spread).to(dtype)
        self.suf = [torch.randn(n, D, generator=g).to(dtype) for n in k_lens]
        self.pre = torch.randn(P, D, generator=g).to(dtype)
        cu = lambda v: torch.tensor([0] + list(np.cumsum(v)), dtype=torch.int32).cuda()  # noqa: E731
        kw, self.prefix = {}, {}
        if page:
            need = [-(-n // page) for n in k_lens + [P]]
            order = torch.randperm(sum(need) + 2, generator=g).tolist()
            kv = torch.full(((sum(need) + 2) * page, D), float("nan"), dtype=dtype)
            table = torch.full((len(k_lens), max(max(need), 1)), -1, dtype=torch.int32)
            for b, rows in enumerate(self.suf + [self.pre]):
                pages = [order.pop() for _ in range(need[b])]
                for i, pg in enumerate(pages):
                    part = rows[i * page:(i + 1) * page]
                    kv[pg * page:pg * page + len(part)] = part
                if b < len(k_lens):
                    table[b, :len(pages)] = torch.tensor(pages, dtype=torch.int32)
                else:
                    self.table = pages
            kw = dict(block_table=table.cuda(), page_size=page, num_pages=sum(need) + 2)
            if P:
                self.prefix = dict(prefix_table=torch.tensor(self.table, dtype=torch.int32).cuda(),
                                   prefix_len=P)
        else:
            kv = torch.cat(self.suf)
            if P:
                self.prefix = dict(prefix_kv=self.pre.cuda())
        self.kv = kv.cuda()
        name = {BF: "bf16", F32: "f32"}[dtype]
        self.prob = dsa.Problem(cu(q_lens), cu(k_lens), q_lens=q_lens, k_lens=k_lens, h_idx=4,
                                d_idx=32, h=h, d_c=d_c, d_rope=d_rope, top_k=8, idx_dtype="f32",
                                kv_dtype=name, **kw)

    def run(self, **kw):
        import sparse_attention_lightning_gb300 as dsa
        return dsa.prefix_mla_attn(self.prob, self.q.cuda(), self.kv, **self.prefix, **kw)

    def rows(self):
        t = 0
        for b, (T, L) in enumerate(zip(self.q_lens, self.k_lens)):
            keys = np.concatenate([self.pre.double().numpy(), self.suf[b].double().numpy()])
            for i in range(T):
                yield t, self.q[t].double().numpy(), keys[:self.P + L - T + i + 1]
                t += 1

    def check(self, out, lse, rows=None):
        """Errors counted, per element.  A logit is off by at most δ = (D + 2) · 2^-24 · max_x scale ·
        Σ_c |q_c k_c| (fp32 accumulation in any order, then the scale), which changes every p by a factor within e^(2δ)
        and lse by δ.  bf16 on the tensor cores: each p is rounded to bf16 (2^-8), the output too (2^-8 of it).
        fp32 sums over n keys: in chains of at most n additions of non-negative p|v|, below 2^-24 · min(n, 4096) of
        Σ p|v| (pieces of a few thousand keys are added up in parallel); 2^-20 for exp2 and the merge of pieces."""
        bf = self.q.dtype == BF
        out, lse = out.float().cpu().double().numpy(), lse.cpu().double().numpy()
        D = self.q.shape[2]
        for t, q, keys in self.rows():
            if rows is not None and t not in rows:
                continue
            ro, rl, mag, top = C.attend(q, keys, self.d_c, self.scale)
            delta = (D + 2) * 2.0 ** -24 * top
            rel = 2 * delta + min(len(keys), 4096) * 2.0 ** -24 + 2.0 ** -20
            tol = rel[:, None] * mag + 1e-30
            if bf:
                tol = tol + 2.0 ** -8 * (mag + np.abs(ro)) * (1 + 2.0 ** -7)
            else:
                tol = tol + 2.0 ** -24 * np.abs(ro)
            err = np.abs(out[t] - ro)
            assert np.all(err <= tol), (t, float((err / tol).max()))
            assert np.all(np.abs(lse[t] - rl) <= rel + 2.0 ** -23 * np.abs(rl)), (t, np.abs(lse[t] - rl).max())


SMALL = dict(d_c=64, d_rope=16)
FULL = dict(d_c=512, d_rope=64)


@pytest.mark.gpu
@pytest.mark.parametrize("page", [0, 16, 64])
@pytest.mark.parametrize("dims", [SMALL, FULL], ids=["64+16", "512+64"])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("q_lens,k_lens,h,P", [
    ([1], [1], 1, 0),                                # one row, one key
    ([1], [1], 128, 1),
    ([1, 1, 1, 1], [1, 63, 64, 65], 16, 100),        # chunk borders in the suffix
    ([1, 1, 1], [5, 200, 7], 128, 64),               # a prefix of whole chunks
    ([3, 1, 0, 17], [3, 130, 4, 300], 20, 129),      # odd heads, an empty sequence, ragged rows
    ([70, 2], [90, 2], 8, 37),                       # prefill chunk: blocks of several tokens
])
def test_matches_definition(q_lens, k_lens, h, P, dims, dtype, page):
    s = Setup(q_lens, k_lens, h, P=P, dtype=dtype, page=page, seed=h + P, spread=2.0, **dims)
    out, lse = s.run()
    s.check(out, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("d_c,d_rope", [(16, 0), (128, 64), (256, 32), (272, 48), (512, 0),
                                        (512, 80), (1024, 256)])
def test_other_widths(d_c, d_rope):
    s = Setup([2, 1], [40, 90], 12, d_c, d_rope, 150, BF, seed=d_c)
    s.check(*s.run())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_long_prefix_split_over_the_card(dtype):
    """Few rows over a long prefix: their keys are cut into pieces and merged."""
    s = Setup([1, 1], [20, 3], 16, P=9001, dtype=dtype, seed=5, spread=3.0, **FULL)
    out, lse = s.run()
    s.check(out, lse)
    out2, lse2 = s.run()
    assert torch.equal(out, out2) and torch.equal(lse, lse2)  # no order of atomics in it


@pytest.mark.gpu
def test_large_logits_move_the_reference():
    """Keys that grow along the sequence: the running max moves by more than 2^8 many times."""
    s = Setup([1], [300], 128, P=500, dtype=BF, seed=6, spread=1.0, **FULL)
    for i, rows in enumerate((s.pre, s.suf[0])):
        rows *= torch.linspace(0.1 + i, 1.0 + 8 * i, len(rows))[:, None].to(BF)
    s.kv = s.suf[0].cuda()
    s.prefix = dict(prefix_kv=s.pre.cuda())
    s.q *= 4
    s.check(*s.run())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,h", [(BF, 128), (BF, 16), (F32, 8)])
def test_nan_and_infinity_in_keys_a_row_does_not_see(dtype, h):
    """A later token's key holds NaN (or infinity): the rows before it are those of clean keys."""
    dims = FULL if dtype == BF else SMALL
    s = Setup([40, 1], [100, 30], h, P=70, dtype=dtype, seed=7, **dims)
    clean = [t.clone() for t in s.suf]
    for bad in (float("nan"), float("inf")):
        s.suf[0] = clean[0].clone()
        s.suf[0][80] = bad                 # position 80: token 20 of sequence 0
        s.kv = torch.cat(s.suf).cuda()
        out, lse = s.run()
        s.suf[0] = clean[0]
        seen = set(range(20, 40))
        s.check(out, lse, rows=set(range(41)) - seen)
        assert torch.isnan(lse[20:40]).any(dim=1).all()


@pytest.mark.gpu
def test_bad_pages_are_reported_and_skipped():
    import sparse_attention_lightning_gb300 as dsa
    for dtype, h in ((F32, 8), (BF, 16)):
        s = Setup([1, 1], [40, 40], h, P=64, dtype=dtype, page=16, seed=8, **SMALL)
        ws = dsa.Workspace()
        ok, lse_ok = s.run(ws=ws)
        assert ws.status() == 0
        s.prob.block_table[1, 1] = 10 ** 6           # keys 16..31 of sequence 1
        out, lse = s.run(ws=ws)
        assert ws.status() == _abi.DSA_FLAG_BAD_INDEX
        assert torch.equal(out[0], ok[0])
        s.suf[1] = torch.cat([s.suf[1][:16], s.suf[1][32:]])
        s.k_lens = [40, 24]
        s.check(out, lse)
        ws.clear_status()
        s.prefix["prefix_table"].fill_(-1)           # no prefix key at all
        s.prob.block_table[1].fill_(-1)
        out, lse = s.run(ws=ws)
        assert ws.status() == _abi.DSA_FLAG_BAD_INDEX
        assert (out[1] == 0).all() and torch.isneginf(lse[1]).all()  # a row without any key


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,h", [(BF, 128), (BF, 16), (F32, 8)])
def test_inconsistent_offsets_are_reported(dtype, h):
    """A sequence whose lengths disagree is skipped; its rows and the others' stay right."""
    import sparse_attention_lightning_gb300 as dsa
    dims = FULL if dtype == BF else SMALL
    s = Setup([2, 2, 1], [30, 30, 30], h, P=40, dtype=dtype, seed=9, **dims)
    out0, lse0 = s.run()
    ws = dsa.Workspace()
    out = torch.full_like(out0, 7.0)
    lse = torch.full_like(lse0, 7.0)
    s.prob.cu_k.copy_(torch.tensor([0, 30, 31, 90], dtype=torch.int32))  # T_1 = 2 > L_1 = 1, L_2 = 59
    s.run(out=out, lse=lse, ws=ws)
    assert ws.status() & _abi.DSA_FLAG_BAD_SEQS
    assert torch.equal(out[:2], out0[:2]) and torch.equal(lse[:2], lse0[:2])
    assert (out[2:] == 7.0).all() and (lse[2:] == 7.0).all()


@pytest.mark.gpu
def test_equals_sparse_attention_while_histories_are_short():
    """Without a prefix, and with every position selected, this is the sparse attention."""
    import sparse_attention_lightning_gb300 as dsa
    from sparse_attention_lightning_gb300 import workloads as W
    cfg = W.custom([1, 30], [90, 64], h_idx=64, d_idx=128, h=128, d_c=512, d_rope=64, top_k=128,
                   idx_dtype="bf16", kv_dtype="bf16")
    case = W.make_case(cfg, 3)
    d = {k: v.cuda() for k, v in case.tensors().items()}
    P = dsa.Problem.from_config(cfg, d["cu_q"], d["cu_k"])
    out, lse, _, _ = dsa.fused_forward(P, d["q_idx"], d["k_idx"], d["w"], d["q"], d["kv"])
    po, pl = dsa.prefix_mla_attn(P, d["q"], d["kv"])
    # each side is within 2^-7 of Σ p|v| (bf16 p and output), and |v| < 6 D^-1/2; the sparse
    # side's fp16 logits add 2^-10 of a logit below 1
    tol = (2 * 2.0 ** -7 + 2.0 ** -9) * 6 * 576 ** -0.5
    assert (out.float() - po.float()).abs().max() <= tol
    assert (lse - pl).abs().max() <= 2e-3


@pytest.mark.gpu
def test_streams_graphs_and_refusals():
    import sparse_attention_lightning_gb300 as dsa
    s = Setup([1, 1, 1], [30, 60, 90], 16, P=2000, dtype=BF, seed=10, **FULL)
    ref, ref_lse = s.run()
    q = s.q.cuda()
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = []
    for st in streams:  # default workspaces belong to a stream: these may overlap
        with torch.cuda.stream(st):
            got.append(dsa.prefix_mla_attn(s.prob, q, s.kv, **s.prefix))
    torch.cuda.synchronize()
    for o, l in got:
        assert torch.equal(o, ref) and torch.equal(l, ref_lse)
    # two graphs with a workspace each, replayed side by side
    graphs = []
    for st in streams[:2]:
        ws = dsa.Workspace(nbytes=s.prob.workspace_size(_abi.OP_PREFIX_MLA_ATTN))
        st.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            o, l = dsa.prefix_mla_attn(s.prob, q, s.kv, ws=ws, **s.prefix)
        graphs.append((graph, o, l, ws))
    q.copy_(q * 0.5)
    torch.cuda.synchronize()
    for st, (graph, *_rest) in zip(streams, graphs):
        with torch.cuda.stream(st):
            graph.replay()
    torch.cuda.synchronize()
    ref, ref_lse = dsa.prefix_mla_attn(s.prob, q, s.kv, **s.prefix)
    for _, o, l, _ws in graphs:
        assert torch.equal(o, ref) and torch.equal(l, ref_lse)
    # a capture that would have to allocate its workspace is refused
    fresh = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with pytest.raises(ValueError):
        with torch.cuda.graph(graph, stream=fresh):
            dsa.prefix_mla_attn(s.prob, q, s.kv, **s.prefix)
    with pytest.raises(ValueError):
        dsa.prefix_mla_attn(s.prob, q, s.kv, prefix_len=5)
    with pytest.raises(ValueError):
        dsa.prefix_mla_attn(s.prob, q, s.kv, prefix_table=torch.zeros(4, dtype=torch.int32).cuda(),
                            prefix_len=5)
    with pytest.raises(ValueError):
        dsa.prefix_mla_attn(s.prob, q, s.kv, prefix_kv=s.pre.cuda(), prefix_len=2001)
    with pytest.raises(ValueError):
        dsa.prefix_mla_attn(s.prob, q[:, :8].contiguous(), s.kv, **s.prefix)


@pytest.mark.gpu
@pytest.mark.parametrize("page", [16, 32, 64, 256])
@pytest.mark.parametrize("dtype,dims", [(BF, FULL), (BF, SMALL), (F32, SMALL)])
def test_packed_prefix_of_a_paged_cache(dtype, dims, page):
    s = Setup([1, 5, 1], [40, 300, 3], 16, P=333, dtype=dtype, page=page, seed=12, **dims)
    s.prefix = dict(prefix_kv=s.pre.cuda())
    s.check(*s.run())


@pytest.mark.gpu
@pytest.mark.parametrize("q_lens,k_lens,h,P", [
    ([1] * 20, [50 + 7 * i for i in range(20)], 128, 4100),  # one key axis, lines cut anywhere
    ([3] * 60, [20] * 60, 20, 4000),                         # blocks over the prefix, and the sequences'
    ([40, 1], [40, 700], 128, 6000),                         # a prefill chunk beside a decode row
    ([0, 200, 0, 1], [5, 333, 1, 64], 128, 3000),            # many blocks of one sequence
])
def test_shares_cut_anywhere(q_lens, k_lens, h, P):
    """Enough work that every SM gets an equal share of the laid-out lines."""
    s = Setup(q_lens, k_lens, h, P=P, dtype=BF, seed=h + P, spread=2.0, **FULL)
    out, lse = s.run()
    n = sum(q_lens)
    s.check(out, lse, rows=set(range(0, n, max(1, n // 12))) | {n - 1})
    again, lse2 = s.run()
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.gpu
def test_a_longer_sequence_than_max_q_len_is_reported():
    import sparse_attention_lightning_gb300 as dsa
    for dtype, h in ((BF, 16), (F32, 8)):
        s = Setup([2, 2], [30, 30], h, P=40, dtype=dtype, seed=13, **SMALL)
        out0, lse0 = s.run()
        ws = dsa.Workspace()
        out, lse = torch.full_like(out0, 7.0), torch.full_like(lse0, 7.0)
        s.prob.cu_q.copy_(torch.tensor([0, 1, 4], dtype=torch.int32))  # T_1 = 3, max_q_len = 2
        s.run(out=out, lse=lse, ws=ws)
        assert ws.status() == _abi.DSA_FLAG_BAD_SEQS and (out[1:] == 7.0).all() and (lse[1:] == 7.0).all()


@pytest.mark.gpu
def test_prefix_len_takes_part_of_the_rows():
    s = Setup([1, 2], [3, 4], 16, P=200, dtype=BF, seed=11, **FULL)
    out, lse = s.run(prefix_len=77)
    s.P, s.pre = 77, s.pre[:77]
    s.check(out, lse)
    out, lse = s.run(prefix_len=0)
    s.P, s.pre = 0, s.pre[:0]
    s.check(out, lse)


@pytest.mark.gpu
def test_a_captured_call_brings_its_workspace():
    """Graphs captured on one stream may be replayed on two, so none may use the stream's own scratch; and
    a workspace that grows later leaves a captured graph the buffer it was captured with."""
    import sparse_attention_lightning_gb300 as dsa
    s = Setup([1, 1], [30, 60], 16, P=2000, dtype=BF, seed=14, **FULL)
    q = s.q.cuda()
    ws = dsa.Workspace(nbytes=s.prob.workspace_size(_abi.OP_PREFIX_MLA_ATTN))
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        ref, ref_lse = dsa.prefix_mla_attn(s.prob, q, s.kv, **s.prefix)  # the stream has its own scratch now
    torch.cuda.synchronize()
    with pytest.raises(ValueError, match="of its own"):
        with torch.cuda.graph(torch.cuda.CUDAGraph(), stream=side):
            dsa.prefix_mla_attn(s.prob, q, s.kv, **s.prefix)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out, lse = dsa.prefix_mla_attn(s.prob, q, s.kv, ws=ws, **s.prefix)
    held = ws.buf.data_ptr()
    big = Setup([1] * 9, [60] * 9, 128, P=2000, dtype=BF, seed=15, **FULL)
    assert big.prob.workspace_size(_abi.OP_PREFIX_MLA_ATTN) > ws.nbytes
    big.check(*big.run(ws=ws), rows={0, 8})
    assert ws.buf.data_ptr() != held
    junk = [torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda") for _ in range(64)]
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ref) and torch.equal(lse, ref_lse)
    assert all((j == 255).all() for j in junk)
