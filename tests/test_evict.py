"""Accumulated attention weight and eviction by it, against the fp64 definitions, and a decode loop
that uses them together with the rest of the layer."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import cache_ops as C
from sparse_attention_lightning_gb300 import _abi

BF, F32 = torch.bfloat16, torch.float32


def test_oracle_keep():
    a = np.array([5.0, 0, 3, 3, 1, 3, 9, 0])
    assert C.keep(a, 8, 0, 0).tolist() == list(range(8))
    assert C.keep(a, 3, 0, 0).tolist() == [0, 2, 6]              # ties: the smaller position
    assert C.keep(a, 4, 2, 1).tolist() == [0, 1, 6, 7]
    assert C.keep(a, 5, 1, 1).tolist() == [0, 2, 3, 6, 7]
    assert C.keep(a, 2, 1, 1).tolist() == [0, 7]


def _problem(**kw):
    base = dict(num_seqs=2, total_q=2, total_k=64, max_q_len=1, max_k_len=40, h_idx=4, d_idx=32,
                h=8, d_c=64, d_rope=16, top_k=8, idx_dtype=2, kv_dtype=1, out_dtype=1,
                sm_scale=0.0, cu_q=4096, cu_k=8192)
    base.update(kw)
    return _abi.DsaProblem(**base)


def test_weights_argument_checks():
    L, A = _abi.lib(), 1 << 20
    bad = _abi.DSA_ERR_INVALID_ARG

    def call(p=None, q=A, kv=A, idx=A, lse=A, acc=A, ld=40, ws=A, wsb=1 << 40):
        return L.dsa_accumulate_attn_weights(ctypes.byref(p or _problem()), q, kv, idx, lse, acc, ld,
                                             ws, wsb, None)

    assert call(q=None) == bad and call(kv=A + 8) == bad and call(idx=None) == bad
    assert call(lse=None) == bad and call(acc=None) == bad and call(acc=A + 2) == bad
    assert call(ld=39) == bad and call(ws=None) == _abi.DSA_ERR_WORKSPACE
    assert call(_problem(max_q_len=2, total_q=4), wsb=16384) == _abi.DSA_ERR_WORKSPACE
    assert call(_problem(kv_dtype=3)) == _abi.DSA_ERR_UNSUPPORTED
    assert call(_problem(total_q=0), q=None, idx=None, lse=None) == _abi.DSA_OK


def test_evict_argument_checks():
    L, A = _abi.lib(), 1 << 24
    bad, unsup = _abi.DSA_ERR_INVALID_ARG, _abi.DSA_ERR_UNSUPPORTED
    paged = dict(page_size=32, max_pages=2, num_pages=4, block_table=1 << 16)

    def call(p=None, acc=A, ld=40, budget=16, sink=2, recent=4, kept=2 * A, cu=3 * A, ao=4 * A,
             ldo=16, kv=5 * A, kvo=6 * A, ki=None, kio=None, ks=None, kso=None, table=None, mp=0,
             np_=0, rows=32, ws=A, wsb=1 << 30):
        return L.dsa_evict(ctypes.byref(p or _problem()), acc, ld, budget, sink, recent, kept, cu,
                           ao, ldo, kv, kvo, ki, kio, ks, kso, table, mp, np_, rows, ws, wsb, None)

    assert call(budget=0) == bad and call(sink=-1) == bad and call(recent=15) == bad
    assert call(acc=None) == bad and call(kept=None) == bad and call(cu=2) == bad
    assert call(ld=39) == bad and call(ldo=15) == bad
    assert call(ao=A + 64) == bad                                  # acc_out over acc
    assert call(kvo=None) == bad and call(ki=7 * A) == bad and call(kso=7 * A) == bad
    assert call(kvo=5 * A) == bad and call(kvo=5 * A + 160) == bad  # a packed move in place
    assert call(kv=5 * A + 8) == bad
    assert call(_problem(idx_dtype=1), ks=7 * A, kso=8 * A) == bad  # scales of keys that have none
    assert call(table=A, mp=1, np_=1) == bad                       # a table without pages
    p = _problem(**paged)
    assert call(p, table=A + 2, mp=1, np_=1) == bad and call(p, table=A, mp=0, np_=1) == bad
    assert call(p, table=A, mp=1, np_=1 << 27) == unsup
    assert call(p, table=A, mp=1, np_=4, kvo=5 * A + 160) == bad    # neither the same pool nor apart
    assert call(rows=-1) == bad
    assert call(cu=8192 + 8) == bad                                # the offsets it reads
    assert call(ws=None) == _abi.DSA_ERR_WORKSPACE and call(wsb=64) == _abi.DSA_ERR_WORKSPACE


# ---------------------------------------------------------------------------
# Accumulated weight.

class Weights:
    def __init__(self, q_lens, k_lens, h, d_c, d_rope, k, dtype, page=0, seed=0, spread=2.0):
        import sparse_attention_lightning_gb300 as dsa
        from sparse_attention_lightning_gb300 import workloads as W
        g = torch.Generator().manual_seed(seed)
        D = d_c + d_rope
        name = {BF: "bf16", F32: "f32"}[dtype]
        cfg = W.custom(q_lens, k_lens, h=h, d_c=d_c, d_rope=d_rope, top_k=k, kv_dtype=name)
        case = W.make_case(cfg, seed)
        case.q = (torch.randn(sum(q_lens), h, D, generator=g) * spread).to(dtype)
        case.kv = torch.randn(sum(k_lens), D, generator=g).to(dtype)
        self.case, self.D, self.scale = case, D, D ** -0.5
        kw, self.kv = {}, case.kv.cuda()
        if page:
            pk = W.paged_keys(case, page, seed)
            self.kv = pk.kv.cuda()
            kw = dict(block_table=pk.block_table.cuda(), page_size=page, num_pages=pk.num_pages)
        self.prob = dsa.Problem.from_config(cfg, case.cu_q.cuda(), case.cu_k.cuda(), **kw)
        self.q = case.q.cuda()
        self.idx = torch.full((sum(q_lens), k), -1, dtype=torch.int32)
        t = 0
        for T, L in zip(q_lens, k_lens):
            for i in range(T):
                n = min(k, L - T + i + 1)
                self.idx[t, :n] = torch.randperm(L - T + i + 1, generator=g)[:n].to(torch.int32)
                t += 1

    def attention(self):
        """The lse of the attention over idx, from its definition, as fp32."""
        cfg = self.case.cfg
        lse = torch.empty(cfg.total_q, cfg.h)
        t = k0 = 0
        for T, L in zip(cfg.q_lens, cfg.k_lens):
            for _ in range(T):
                i = self.idx[t][(self.idx[t] >= 0) & (self.idx[t] < L)]
                lse[t] = torch.from_numpy(C.attend(self.case.q[t].double().numpy(),
                                                   self.case.kv[k0 + i.long()].double().numpy(),
                                                   cfg.d_c, self.scale)[1])
                t += 1
            k0 += L
        return lse.cuda()

    def reference(self, lse, acc):
        """(acc + weights, their error bound): a logit is off by (D + 2) · 2^-24 · scale · Σ|q_c k_c|,
        the exponent's argument by 2^-23 of |logit| and |lse| more, the sum over heads by H · 2^-24, exp2 by
        2^-21; then one fp32 rounding a query (or 2^-40 in fixed point) and one of the sum."""
        cfg = self.case.cfg
        out, tol = acc.double().cpu().numpy(), np.zeros(acc.shape)
        q, kv = self.case.q.double().numpy(), self.case.kv.double().numpy()
        ls = lse.double().cpu().numpy()
        t = k0 = 0
        for b, (T, L) in enumerate(zip(cfg.q_lens, cfg.k_lens)):
            for _ in range(T):
                i = self.idx[t].numpy()
                i = i[(i >= 0) & (i < L)]
                keys = kv[k0 + i]
                w = C.weights(q[t], keys, ls[t], self.scale)
                mag = (np.abs(q[t]) @ np.abs(keys).T).max(axis=0) * self.scale
                top = np.abs(ls[t][np.isfinite(ls[t])]).max(initial=0.0)
                rel = (self.D + 2) * 2.0 ** -24 * mag + 2.0 ** -22 * (mag + top) + cfg.h * 2.0 ** -24 + 2.0 ** -20
                np.add.at(out[b], i, w)
                np.add.at(tol[b], i, w * rel)
                t += 1
            k0 += L
        return out, tol + 2.0 ** -22 * np.abs(out) + 2.0 ** -40 * cfg.total_q

    def check(self, lse=None, acc=None):
        import sparse_attention_lightning_gb300 as dsa
        cfg = self.case.cfg
        lse = self.attention() if lse is None else lse
        if acc is None:
            acc = torch.rand(cfg.num_seqs, max(cfg.k_lens) + 5).cuda()
        ref, tol = self.reference(lse, acc)
        before = acc.clone()
        got = dsa.accumulate_attn_weights(self.prob, self.q, self.kv, self.idx.cuda(), lse, acc)
        assert got.data_ptr() == acc.data_ptr()
        err = np.abs(got.double().cpu().numpy() - ref)
        assert np.all(err <= tol), float((err / tol).max())
        for b, L in enumerate(cfg.k_lens):  # columns behind a sequence stay as they were
            assert torch.equal(acc[b, L:], before[b, L:])
        return before, lse, got


@pytest.mark.gpu
@pytest.mark.parametrize("page", [0, 16])
@pytest.mark.parametrize("dtype,h,d_c,d_rope", [(F32, 8, 64, 16), (BF, 20, 64, 16), (BF, 128, 512, 64),
                                                (BF, 1, 16, 0), (BF, 100, 512, 0), (BF, 7, 1024, 256)])
@pytest.mark.parametrize("q_lens,k_lens,k", [
    ([1], [1], 1), ([1, 1, 1], [700, 3, 130], 200), ([5, 0, 1, 33], [5, 9, 64, 129], 40)])
def test_weights_match_definition(q_lens, k_lens, k, dtype, h, d_c, d_rope, page):
    s = Weights(q_lens, k_lens, h, d_c, d_rope, k, dtype, page, seed=h + k)
    before, lse, got = s.check()
    # every query's probabilities add up to its heads (their sum over all positions)
    added = float(got.double().sum() - before.double().sum())
    want = h * sum(q_lens)
    assert abs(added - want) <= 1e-3 * want


@pytest.mark.gpu
def test_weights_repeats_padding_and_empty_heads():
    """Repeated and skipped entries, heads without an lse, and the same bytes on every run."""
    import sparse_attention_lightning_gb300 as dsa
    for q_lens in ([1, 1], [9, 30]):
        s = Weights(q_lens, [50, 60], 16, 64, 16, 24, BF, seed=3)
        s.idx[0, :8] = 4
        s.idx[:, 20:] = -1
        lse = s.attention()
        lse[1, 3:9] = -float("inf")
        before, _, got = s.check(lse=lse)
        again = dsa.accumulate_attn_weights(s.prob, s.q, s.kv, s.idx.cuda(), lse, before.clone())
        assert torch.equal(got, again)
        ws = dsa.Workspace()
        s.idx[0, 9] = 10 ** 6
        s.idx[0, 10] = -7
        ref, tol = s.reference(lse, before)
        bad = dsa.accumulate_attn_weights(s.prob, s.q, s.kv, s.idx.cuda(), lse, before.clone(), ws=ws)
        assert ws.status() == _abi.DSA_FLAG_BAD_INDEX


@pytest.mark.gpu
def test_checked_build_raises_no_flag():
    """The kernels' own checks of gather rows and accumulator slots, in the build that has them."""
    import sparse_attention_lightning_gb300 as dsa
    from sparse_attention_lightning_gb300 import build
    build.build(checked=True)
    for q_lens, dtype, page in (([1, 1], BF, 0), ([4, 9], BF, 16), ([4, 9], F32, 0)):
        s = Weights(q_lens, [200, 90], 16, 64, 16, 50, dtype, page, seed=6)
        lse = s.attention()
        ref = dsa.accumulate_attn_weights(s.prob, s.q, s.kv, s.idx.cuda(), lse, torch.zeros(2, 200).cuda())
        ws = dsa.Workspace()
        with _abi.using(_abi.CHECKED_LIB_PATH):
            got = dsa.accumulate_attn_weights(s.prob, s.q, s.kv, s.idx.cuda(), lse,
                                              torch.zeros(2, 200).cuda(), ws=ws)
            assert ws.status() == 0
        assert torch.equal(got, ref)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
def test_weights_inconsistent_offsets_are_reported(dtype):
    import sparse_attention_lightning_gb300 as dsa
    s = Weights([2, 2, 1], [40, 50, 9], 16, 64, 16, 64, dtype, seed=5)
    lse = s.attention()
    ref = dsa.accumulate_attn_weights(s.prob, s.q, s.kv, s.idx.cuda(), lse, torch.zeros(3, 50).cuda())
    ws = dsa.Workspace()
    s.prob.cu_q.copy_(torch.tensor([0, 2, 5, 5], dtype=torch.int32))  # 3 queries, max_q_len = 2
    got = dsa.accumulate_attn_weights(s.prob, s.q, s.kv, s.idx.cuda(), lse, torch.zeros(3, 50).cuda(), ws=ws)
    assert ws.status() == _abi.DSA_FLAG_BAD_SEQS
    assert torch.equal(got[0], ref[0]) and (got[1:] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("q_lens", [[1, 1], [2, 3]])
def test_weights_nan_reaches_only_its_position(q_lens):
    import sparse_attention_lightning_gb300 as dsa
    s = Weights(q_lens, [40, 50], 16, 64, 16, 64, BF, seed=4)
    lse = s.attention()
    acc0 = torch.zeros(2, 50).cuda()
    ref = dsa.accumulate_attn_weights(s.prob, s.q, s.kv, s.idx.cuda(), lse, acc0.clone())
    s.kv[7] = float("nan")  # position 7 of sequence 0
    got = dsa.accumulate_attn_weights(s.prob, s.q, s.kv, s.idx.cuda(), lse, acc0.clone())
    assert torch.isnan(got[0, 7])
    ref[0, 7] = got[0, 7] = 0
    assert torch.equal(got, ref)


# ---------------------------------------------------------------------------
# Eviction.

def _caches(k_lens, idx_dtype, page, seed, budget, d_c=64, d_rope=16, d_idx=64):
    """(problem, caches, destination) with every cache row distinct."""
    import sparse_attention_lightning_gb300 as dsa
    from sparse_attention_lightning_gb300 import workloads as W
    cfg = W.custom([0] * len(k_lens), k_lens, d_c=d_c, d_rope=d_rope, d_idx=d_idx,
                   idx_dtype=idx_dtype, kv_dtype="bf16")
    case = W.make_case(cfg, seed)
    keys = dict(kv=case.kv, k_idx=case.k_idx)
    if case.k_scale is not None:
        keys["k_scale"] = case.k_scale
    kw, out, place = {}, {}, dict(keys)
    n = [min(L, budget) for L in k_lens]
    if page:
        pk = W.paged_keys(case, page, seed)
        kw = dict(block_table=pk.block_table.cuda(), page_size=page, num_pages=pk.num_pages)
        place = {k: getattr(pk, k) for k in keys}
        need = [-(-m // page) for m in n]
        order = torch.randperm(sum(need) + 1, generator=torch.Generator().manual_seed(seed))
        table = torch.full((len(n), max(need)), -1, dtype=torch.int32)
        at = 0
        for b, m in enumerate(need):
            table[b, :m] = order[at:at + m].to(torch.int32)
            at += m
        out["block_table_out"] = table.cuda()
        for k, v in keys.items():
            out[k + "_out"] = torch.full(((sum(need) + 1) * page,) + tuple(v.shape[1:]), 77,
                                         dtype=v.dtype).cuda()
    P = dsa.Problem.from_config(cfg, case.cu_q.cuda(), case.cu_k.cuda(), **kw)
    return P, keys, {k: v.cuda() for k, v in place.items()}, out


def _check_eviction(P, keys, r, out, acc, budget, sink, recent, page):
    k0, used = 0, {k: np.zeros(len(v), bool) for k, v in (("kv", r.kv),)}
    cu = [0]
    for b, L in enumerate(P.k_lens):
        want = C.keep(acc[b, :L].double().cpu().numpy(), budget, sink, recent)
        m = len(want)
        kept = r.kept[b].cpu().numpy()
        assert np.array_equal(kept[:m], want) and np.all(kept[m:] == -1), b
        a = r.acc[b].cpu()
        assert torch.equal(a[:m], acc[b].cpu()[want]) and (a[m:] == 0).all()
        slot = torch.arange(m)
        if page:
            rows = out["block_table_out"][b].cpu()[slot // page].long() * page + slot % page
        else:
            rows = cu[-1] + slot
        used["kv"][rows] = True
        for k, src in keys.items():
            assert torch.equal(getattr(r, k).cpu()[rows].float(), src[k0 + want].float()), (b, k)
        cu.append(cu[-1] + m)
        k0 += L
    assert r.cu_k.cpu().tolist() == cu and r.k_lens == np.diff(cu).tolist()
    if page:  # rows that hold no kept position stay as they were
        for k in keys:
            assert (getattr(r, k).cpu()[~used["kv"]] == 77).all()


@pytest.mark.gpu
@pytest.mark.parametrize("page", [0, 16, 64])
@pytest.mark.parametrize("idx_dtype", ["e4m3", "mxfp8", "bf16"])
@pytest.mark.parametrize("k_lens,budget,sink,recent", [
    ([1], 1, 0, 0), ([1, 40, 17], 100, 3, 5), ([50, 200, 64], 64, 0, 0), ([3000, 1, 65, 1024], 65, 60, 5),
    ([5000, 1025, 999], 1000, 7, 40), ([60000, 49153, 31], 20000, 5, 9), ([2100], 1, 1, 0), ([130, 129], 128, 0, 128)])
def test_evict_matches_definition(k_lens, budget, sink, recent, idx_dtype, page):
    import sparse_attention_lightning_gb300 as dsa
    P, keys, caches, out = _caches(k_lens, idx_dtype, page, seed=budget, budget=budget)
    g = torch.Generator().manual_seed(budget + 1)
    acc = torch.rand(len(k_lens), max(k_lens) + 3, generator=g)
    acc = (acc * 50).floor() / 7  # many equal values: ties
    acc = acc.cuda()
    keep_src = {k: v.clone() for k, v in caches.items()}
    r = dsa.evict(P, acc, budget, sink, recent, **caches, **out)
    for k, v in keep_src.items():
        assert torch.equal(caches[k].float().nan_to_num(), v.float().nan_to_num())
    _check_eviction(P, keys, r, out, acc, budget, sink, recent, page)


@pytest.mark.gpu
@pytest.mark.parametrize("fill", ["equal", "negative", "spread", "special"])
def test_evict_values(fill):
    """Equal, negative and widely spread weights, infinities, signed zeros."""
    import sparse_attention_lightning_gb300 as dsa
    P, keys, caches, out = _caches([3001, 700], "e4m3", 0, seed=2, budget=600)
    g = torch.Generator().manual_seed(1)
    acc = torch.randn(2, 3001, generator=g)
    if fill == "equal":
        acc[:] = 0.25
    elif fill == "spread":
        acc = torch.exp(40 * acc)
    elif fill == "special":
        acc[0, 100:900] = float("inf")
        acc[0, 1000:1400] = -0.0
        acc[0, 1400:1800] = 0.0
        acc[1] = -float("inf")
    acc = acc.cuda()
    r = dsa.evict(P, acc, 600, 10, 20, **caches)
    _check_eviction(P, keys, r, out, acc, 600, 10, 20, 0)


@pytest.mark.gpu
def test_evict_strided_acc_and_parts():
    """A strided accumulator, a wider acc_out, and a call that moves nothing."""
    import sparse_attention_lightning_gb300 as dsa
    P, keys, caches, out = _caches([300, 80], "e4m3", 0, seed=5, budget=100)
    acc = torch.rand(2, 777).cuda()[:, 11:411]
    wide = torch.full((2, 160), 5.0).cuda()
    r = dsa.evict(P, acc, 100, 1, 2, kv=caches["kv"], acc_out=wide)
    assert r.k_idx is None and r.acc is wide
    assert (wide[:, 100:] == 5.0).all()  # columns past the budget stay as they were
    _check_eviction(P, {"kv": keys["kv"]}, r._replace(acc=wide[:, :100]), out, acc, 100, 1, 2, 0)
    part = torch.full((2, 130), 5.0).cuda()  # a part of wider rows
    r = dsa.evict(P, acc, 100, 1, 2, acc_out=part[:, 20:120])
    assert (part[:, :20] == 5.0).all() and (part[:, 120:] == 5.0).all()
    assert torch.equal(r.acc, wide[:, :100])
    r = dsa.evict(P, acc, 100)
    assert r.kv is None and r.kept[1, 80:].eq(-1).all()
    with pytest.raises(ValueError):
        dsa.evict(P, acc, 100, 60, 41)
    with pytest.raises(ValueError):
        dsa.evict(P, acc, 100, kv_out=caches["kv"])
    with pytest.raises(ValueError):
        dsa.evict(P, acc[:, :200], 100)
    with pytest.raises(ValueError):
        dsa.evict(P, acc, 100, kv=caches["kv"], kv_out=caches["kv"][:179].clone())
    with pytest.raises(_abi.DsaError):
        dsa.evict(P, acc, 100, kv=caches["kv"], kv_out=caches["kv"])


@pytest.mark.gpu
def test_evict_within_one_pool_and_bad_pages():
    """Source and destination pages of the same pool; pages outside it are reported."""
    import sparse_attention_lightning_gb300 as dsa
    from sparse_attention_lightning_gb300 import workloads as W
    cfg = W.custom([0, 0], [200, 90], d_c=64, d_rope=16, d_idx=64, idx_dtype="e4m3", kv_dtype="bf16")
    case = W.make_case(cfg, 6)
    pk = W.paged_keys(case, 16, 6, spare_pages=12)
    used = set(pk.block_table[pk.block_table >= 0].tolist())
    free = [p for p in range(pk.num_pages) if p not in used]
    table = torch.tensor([free[:5], free[5:10]], dtype=torch.int32).cuda()
    pool = {k: getattr(pk, k).cuda() for k in ("kv", "k_idx", "k_scale")}
    P = dsa.Problem.from_config(cfg, case.cu_q.cuda(), case.cu_k.cuda(), block_table=pk.block_table.cuda(),
                                page_size=16, num_pages=pk.num_pages)
    acc = torch.rand(2, 200).cuda()
    outs = {k + "_out": v for k, v in pool.items()}
    r = dsa.evict(P, acc, 80, 2, 3, **pool, **outs, block_table_out=table)
    for b, (L, k0) in enumerate(((200, 0), (90, 200))):
        want = C.keep(acc[b, :L].double().cpu().numpy(), 80, 2, 3)
        rows = table[b].cpu()[torch.arange(80) // 16].long() * 16 + torch.arange(80) % 16
        assert torch.equal(r.kv.cpu()[rows], case.kv[k0 + want])
    ws = dsa.Workspace()
    table[1, 2] = pk.num_pages
    before = pool["kv"].clone()
    dsa.evict(P, acc, 80, 2, 3, **pool, **outs, block_table_out=table, ws=ws)
    assert ws.status() == _abi.DSA_FLAG_BAD_SEQS and torch.equal(pool["kv"], before)


@pytest.mark.gpu
def test_evict_graph_and_streams():
    import sparse_attention_lightning_gb300 as dsa
    P, keys, caches, out = _caches([900, 400], "e4m3", 0, seed=7, budget=300)
    acc = torch.rand(2, 900).cuda()
    ws = dsa.Workspace()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = dsa.evict(P, acc, 300, 5, 50, **caches, ws=ws)
    acc.copy_(torch.rand(2, 900))
    graph.replay()
    torch.cuda.synchronize()
    _check_eviction(P, keys, r, out, acc, 300, 5, 50, 0)


# ---------------------------------------------------------------------------
# Together: keys normalised and quantised, selected, attended, weighed, evicted, attended again.

@pytest.mark.gpu
@pytest.mark.parametrize("quant", ["e4m3", "mxfp8"])
def test_a_layer_that_evicts(quant):
    import sparse_attention_lightning_gb300 as dsa
    from oracle import dsa_oracle as O
    from sparse_attention_lightning_gb300 import workloads as W
    dims = dict(h_idx=64, d_idx=128, h=128, d_c=512, d_rope=64, top_k=256)
    cfg = W.custom([1, 1, 1], [900, 300, 2000], idx_dtype=quant, kv_dtype="bf16", **dims)
    case = W.make_case(cfg, 8)
    d = {k: v.cuda() for k, v in case.tensors().items()}
    # the index keys: a projection's output, normalised and quantised
    proj = torch.randn(cfg.total_k, 128, generator=torch.Generator().manual_seed(1)).to(BF).cuda()
    gamma = torch.full((128,), 0.1, dtype=BF, device="cuda")
    _, _, k_idx, k_scale = dsa.add_rmsnorm(proj, gamma, quant=quant)
    P = dsa.Problem.from_config(cfg, d["cu_q"], d["cu_k"])
    out, lse, idx, _ = dsa.fused_forward(P, d["q_idx"], k_idx, d["w"], d["q"], d["kv"], d["q_scale"], k_scale)
    acc = torch.zeros(3, P.max_k_len, device="cuda")
    dsa.accumulate_attn_weights(P, d["q"], d["kv"], idx, lse, acc)
    # all weight lies on the selected positions, H of it a query (the attention's fp16 logits: 1e-2)
    assert (acc.sum(dim=1) - 128).abs().max() <= 1.28
    for b in range(3):
        sel = idx[b][idx[b] >= 0].long()
        rest = torch.ones(P.max_k_len, dtype=torch.bool, device="cuda")
        rest[sel] = False
        assert (acc[b][rest] == 0).all() and (acc[b][sel] > 0).all()
    r = dsa.evict(P, acc, 400, sink=4, recent=32, kv=d["kv"], k_idx=k_idx, k_scale=k_scale)
    assert r.k_lens == [400, 300, 400]
    # the smaller caches, through the layer again: the oracle on the same rows
    small = W.custom([1, 1, 1], r.k_lens, idx_dtype=quant, kv_dtype="bf16", **dims)
    P2 = dsa.Problem.from_config(small, d["cu_q"], r.cu_k)
    o2, l2, i2, _ = dsa.fused_forward(P2, d["q_idx"], r.k_idx, d["w"], d["q"], r.kv, d["q_scale"], r.k_scale)
    c2 = W.Case(small, case.cu_q, r.cu_k.cpu(), case.q_idx, r.k_idx.cpu(), case.w, case.q, r.kv.cpu(),
                case.q_scale, r.k_scale.cpu())
    from parity import check_attn_row, check_topk_row, tol_for
    ref = O.problem_from_case(c2)
    for t in range(3):
        sel = i2[t][i2[t] >= 0].cpu().numpy()
        check_topk_row(i2[t].cpu().numpy(), ref.scores(t), 256)
        ro, rl = ref.sfa(t, sel)
        check_attn_row(o2[t].float().cpu().numpy(), l2[t].cpu().numpy(), ro, rl, tol_for(small), f"row {t}")
    # nothing that carried weight was lost: keeping every selected position keeps the output
    kept = [set(r.kept[b][r.kept[b] >= 0].tolist()) for b in range(3)]
    assert all(set(idx[b][idx[b] >= 0].tolist()) <= kept[b] for b in range(3))
    # while a cache holds no more positions than top_k, dense and sparse attention agree
    dense, dl = dsa.prefix_mla_attn(P2, d["q"], r.kv)
    assert (dl - l2).min() >= -2e-3  # the dense sum has every key


@pytest.mark.gpu
@pytest.mark.parametrize("page,q_lens", [(0, [1, 1, 1]), (64, [2, 1, 2])])
def test_kernels_behind_one_another(page, q_lens):
    """Each operator right behind the one that writes its input, no wait between them on the host, in a stream and as
    a captured graph that joins a copy on another stream: the same bytes as with a device-wide wait after each."""
    import sparse_attention_lightning_gb300 as dsa
    from sparse_attention_lightning_gb300 import workloads as W
    dims = dict(h_idx=64, d_idx=128, h=128, d_c=512, d_rope=64, top_k=256)
    cfg = W.custom(q_lens, [900, 300, 2000], idx_dtype="e4m3", kv_dtype="bf16", **dims)
    d = {k: v.cuda() for k, v in W.make_case(cfg, 8).tensors().items()}
    g = torch.Generator().manual_seed(3)
    kw, rows = {}, cfg.total_k
    if page:
        n = [-(-L // page) for L in cfg.k_lens]
        order = torch.randperm(sum(n), generator=g).to(torch.int32)
        table = torch.full((3, max(n)), -1, dtype=torch.int32)
        for b in range(3):
            table[b, :n[b]] = order[sum(n[:b]):sum(n[:b + 1])]
        kw, rows = dict(block_table=table.cuda(), page_size=page, num_pages=sum(n)), sum(n) * page
    P = dsa.Problem.from_config(cfg, d["cu_q"], d["cu_k"], **kw)
    kv0 = (torch.randn(rows, 576, generator=g) / 24).to(BF).cuda()
    proj0 = torch.randn(rows, 128, generator=g).to(BF).cuda()
    prompt = (torch.randn(500, 576, generator=g) / 24).to(BF).cuda()
    gamma, wide = torch.full((128,), 0.1, dtype=BF).cuda(), torch.full((576,), 0.04, dtype=BF).cuda()
    small = W.custom(q_lens, [min(L, 400) for L in cfg.k_lens], idx_dtype="e4m3", kv_dtype="bf16", **dims)
    cu_small = torch.zeros(4, dtype=torch.int32, device="cuda")
    P2 = dsa.Problem.from_config(small, d["cu_q"], cu_small)
    ws = [dsa.Workspace(nbytes=n) for n in (P.workspace_size(_abi.OP_FUSED_FORWARD), P.workspace_size(_abi.OP_ATTN_WEIGHTS),
                                            16384, P2.workspace_size(_abi.OP_PREFIX_MLA_ATTN))]
    kv, proj = kv0.clone(), proj0.clone()

    def step(i, wait):
        proj.copy_(proj0).mul_(1 + i)
        _, _, k_idx, k_scale = dsa.add_rmsnorm(proj, gamma, quant="e4m3")
        wait()
        y, kv_new, _, _ = dsa.add_rmsnorm(kv, wide, residual=kv0)
        wait()
        out, lse, idx, _ = dsa.fused_forward(P, d["q_idx"], k_idx, d["w"], d["q"], y, d["q_scale"], k_scale, ws=ws[0])
        wait()
        acc = torch.zeros(3, P.max_k_len, device="cuda")
        dsa.accumulate_attn_weights(P, d["q"], y, idx, lse, acc, ws=ws[1])
        wait()
        r = dsa.evict(P, acc, 400, sink=4, recent=32, kv=y, k_idx=k_idx, k_scale=k_scale, cu_k_out=cu_small,
                      ws=ws[2]) if not page else None
        wait()
        if r is None:
            out2, lse2 = dsa.prefix_mla_attn(P, d["q"], y, prompt, ws=ws[3])
        else:
            out2, lse2 = dsa.prefix_mla_attn(P2, d["q"], r.kv, prompt, ws=ws[3])
        wait()
        # the output's rows, normalised by the next launch
        y2, _, _, _ = dsa.add_rmsnorm(out2, wide[:512])
        kv.copy_(kv_new)
        wait()
        return [k_idx, k_scale, out, lse, idx, acc, out2, lse2, y2] + ([] if r is None else [r.kept, r.kv, r.acc])

    def same(got, want):
        return all(torch.equal(x.view(torch.uint8) if x.element_size() == 1 else x,
                               y.view(torch.uint8) if y.element_size() == 1 else y) for x, y in zip(got, want))

    want = [step(i, torch.cuda.synchronize) for i in range(6)]
    kv.copy_(kv0)
    got = [step(i, lambda: None) for i in range(6)]
    torch.cuda.synchronize()
    assert all(same(x, y) for x, y in zip(got, want))
    assert not torch.equal(want[0][8], want[1][8])  # the steps differ
    # captured, behind a copy on a stream that joins
    kv.zero_()
    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main):
        side.wait_stream(main)
        with torch.cuda.stream(side):
            kv.copy_(kv0)
        main.wait_stream(side)
        got = [step(i, lambda: None) for i in range(2)]
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert all(same(x, y) for x, y in zip(got, want))
    assert all(w.status() == 0 for w in ws)
