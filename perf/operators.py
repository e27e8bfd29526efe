"""What the operators around the DSA caches cost: the residual RMS norm with 8-bit outputs, dense MLA
attention over a prefix a batch shares, the accumulated attention weight of cached positions, and
the eviction of positions by it.

`run` computes an operator in elementary torch operations (own = False) or through the
framework's call (own = True), on the same state.
"""
import math
import random

import torch

own = False

LOG2E = 1.4426950408889634


# ---------------------------------------------------------------------------
# Cases.

def listed():
    return [
        # one decoded token's hidden state (the prolog's d_model) ahead of a layer: latency only
        dict(name="norm, one token", op="norm", rows=1, d=7168, dtype="bf16", residual=True,
             quant="none", stride=0),
        # the hidden states of an 8k prefill: normalised for the next layer, residual kept
        dict(name="norm, 8k prefill", op="norm", rows=8192, d=7168, dtype="bf16", residual=True,
             quant="none", stride=0),
        # indexer keys of 64k tokens on their way into an MXFP8 key cache, a slice of a wider
        # projection's output
        dict(name="norm, index keys mxfp8", op="norm", rows=65536, d=128, dtype="bf16",
             residual=False, quant="mxfp8", stride=704),
        # a ragged fp32 batch with per-row E4M3 codes: odd row length, no vector loads
        dict(name="norm, odd fp32 e4m3", op="norm", rows=517, d=5001, dtype="f32", residual=True,
             quant="e4m3", stride=0),
        # four samples of a short prompt, 16 heads a GPU: the smallest attention, latency only
        dict(name="prefix, 4 samples", op="prefix", B=4, heads=16, d_c=512, d_rope=64, prefix=1000,
             t_max=1, s_max=61, page=0, dtype="bf16", lens_seed=1),
        # 32 decode rows with all 128 heads behind one 32k system prompt: tensor-core bound
        dict(name="prefix, 32 rows 32k", op="prefix", B=32, heads=128, d_c=512, d_rope=64,
             prefix=32768, t_max=1, s_max=512, page=0, dtype="bf16", lens_seed=2),
        # speculative steps of 64 sequences with 16 heads, paged cache, prefix ends inside a page
        dict(name="prefix, paged 16 heads", op="prefix", B=64, heads=16, d_c=512, d_rope=64,
             prefix=12345, t_max=4, s_max=700, page=64, dtype="bf16", lens_seed=3),
        # the fp32 shape of the tiny workload: ragged prefill chunks behind a shared prefix
        dict(name="prefix, fp32 chunks", op="prefix", B=3, heads=8, d_c=64, d_rope=16, prefix=256,
             t_max=40, s_max=130, page=0, dtype="f32", lens_seed=4),
        # one decode step of the 32-sequence workload: weights of 2048 selected positions a row
        dict(name="weights, decode", op="weights", B=32, heads=128, d_c=512, d_rope=64, t_max=1,
             l_min=8192, l_max=32768, top_k=2048, page=0, dtype="bf16", lens_seed=5),
        # prefill chunks: several queries of a sequence add to the same positions
        dict(name="weights, chunks", op="weights", B=2, heads=128, d_c=512, d_rope=64, t_max=75,
             l_min=200, l_max=1100, top_k=500, page=64, dtype="bf16", lens_seed=6),
        # the 32-sequence workload's caches cut to 8192 positions each, FP8 index keys, paged
        dict(name="evict, 32 caches", op="evict", B=32, d_c=512, d_rope=64, l_min=8192,
             l_max=32768, budget=8192, sink=64, recent=512, page=64, lens_seed=7),
        # one short packed cache: latency
        dict(name="evict, one cache", op="evict", B=1, d_c=512, d_rope=64, l_min=1999, l_max=1999,
             budget=500, sink=4, recent=33, page=0, lens_seed=8),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(("norm", "prefix", "prefix", "weights", "evict"))
    if op == "norm":
        rows = _log(rng, 1, 65536)
        quant = rng.choice(("none", "e4m3", "mxfp8"))
        dtype = rng.choice(("bf16", "bf16", "f32"))
        d = _log(rng, 32, min(8192, max(32, 8192 * (7168 if dtype == "bf16" else 4800) // rows)))
        if quant == "mxfp8":
            d = d // 32 * 32
        elif rng.random() < 0.6:
            d = max(8, d // 8 * 8)
        residual = rng.random() < 0.5
        return dict(op=op, rows=rows, d=d, dtype=dtype, residual=residual, quant=quant,
                    stride=0 if residual or rng.random() < 0.5 else d + 8 * rng.randint(1, 40))
    page = rng.choice((0, 16, 64, 256))
    seed = rng.randint(1, 1 << 20)
    if op == "prefix":
        f32 = rng.random() < 0.15
        d_c, d_rope = (64, 16) if f32 else rng.choice(((512, 64), (512, 64), (512, 64), (256, 32),
                                                       (64, 16), (512, 0), (128, 64)))
        B = _log(rng, 1, 64)
        t_max = rng.choice((1, 1, 1, 2, 5, rng.randint(6, 60)))
        heads = rng.choice((1, 8, 16, 20, 64, 128))
        s_max = max(t_max, _log(rng, 1, 900))
        room = 32 * 128 * 32768 // (B * t_max * heads) // (8 if f32 else 1) // (8 if t_max > 5 else 1)
        P = min(_log(rng, 1, 32768), room) if rng.random() < 0.9 else 0
        return dict(op=op, B=B, heads=heads, d_c=d_c, d_rope=d_rope, prefix=P, t_max=t_max,
                    s_max=min(s_max, max(t_max, 200)) if t_max > 5 else s_max, page=page,
                    dtype="f32" if f32 else "bf16", lens_seed=seed)
    if op == "weights":
        B, t_max = _log(rng, 1, 32), rng.choice((1, 1, 1, 3, rng.randint(4, 32)))
        l_max = max(t_max, _log(rng, 10, 32768))
        top_k = min(_log(rng, 1, 2048), 65536 // (B * t_max))
        f32 = rng.random() < 0.15
        d_c, d_rope = (64, 16) if f32 else rng.choice(((512, 64), (512, 64), (256, 32), (64, 16)))
        return dict(op=op, B=B, heads=rng.choice((8, 16, 20, 64, 128)), d_c=d_c, d_rope=d_rope,
                    t_max=t_max, l_min=max(t_max, l_max // 4), l_max=l_max, top_k=max(1, top_k),
                    page=page, dtype="f32" if f32 else "bf16", lens_seed=seed)
    l_max = _log(rng, 20, 32768)
    budget = _log(rng, 1, l_max)
    sink = rng.randint(0, min(64, budget // 3))
    return dict(op=op, B=_log(rng, 1, 32), d_c=512, d_rope=64, l_min=max(1, l_max // 4),
                l_max=l_max, budget=min(budget, 8192), sink=sink,
                recent=rng.randint(0, min(512, min(budget, 8192) - sink)), page=page, lens_seed=seed)


def _lens(case):
    """(q_lens, k_lens) of a case, from the case alone."""
    r = random.Random(case["lens_seed"])
    if case["op"] == "evict":
        return [0] * case["B"], [r.randint(case["l_min"], case["l_max"]) for _ in range(case["B"])]
    T = case["t_max"]
    q = [T if r.random() < 0.5 else r.randint(1, T) for _ in range(case["B"])]
    if case["op"] == "prefix":
        return q, [r.randint(t, case["s_max"]) for t in q]
    return q, [r.randint(max(t, case["l_min"]), case["l_max"]) for t in q]


def _pairs(case):
    """(query, key) pairs: with the prefix and the suffixes, or the selected ones."""
    q, k = _lens(case)
    if case["op"] == "prefix":
        return sum(t * case["prefix"] + t * (L - t) + t * (t + 1) // 2 for t, L in zip(q, k))
    return sum(min(case["top_k"], L - t + i + 1) for t, L in zip(q, k) for i in range(t))


def work(case):
    op = case["op"]
    if op == "norm":
        n, b = case["rows"] * case["d"], 2 if case["dtype"] == "bf16" else 4
        per = b * (3 if case["residual"] else 1)
        out = b * n if case["quant"] == "none" else n
        sc = {"none": 0, "e4m3": 4 * case["rows"], "mxfp8": n // 32}[case["quant"]]
        return {"bytes": n * per + out + sc + b * case["d"], "flops": 6 * n}
    q, k = _lens(case)
    D = case["d_c"] + case["d_rope"]
    if op == "evict":
        n = sum(min(L, case["budget"]) for L in k)
        return {"bytes": 4 * sum(k) + 2 * n * (D * 2 + 128 + 4 + 4) + 4 * n, "flops": 2 * sum(k)}
    b, H, TQ = 2 if case["dtype"] == "bf16" else 4, case["heads"], sum(q)
    if op == "prefix":
        return {"bytes": b * D * (case["prefix"] + sum(k)) + TQ * H * (b * (D + case["d_c"]) + 4),
                "flops": 2 * H * (D + case["d_c"]) * _pairs(case)}
    n = _pairs(case)
    seen = min(n, sum(k))
    return {"bytes": b * D * seen + 8 * seen + 4 * TQ * case["top_k"] + TQ * H * (b * D + 4),
            "flops": 2 * H * D * n}


# ---------------------------------------------------------------------------
# Inputs.

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
DEV = "cuda"


def _randn(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)


def _offsets(lens):
    c = [0]
    for n in lens:
        c.append(c[-1] + n)
    return torch.tensor(c, dtype=torch.int32, device=DEV)


def _pages(lens, page, g):
    """A block table over a pool of pages in a random order with three spare pages."""
    need = [-(-n // page) for n in lens]
    order = torch.randperm(sum(need) + 3, generator=g, device=DEV).to(torch.int32)
    per = torch.tensor(need, device=DEV)
    first = torch.cumsum(per, 0) - per
    slot = torch.arange(max(max(need), 1), device=DEV)
    at = (first[:, None] + slot[None]).clamp(max=len(order) - 1)
    table = torch.where(slot[None] < per[:, None], order[at], torch.full_like(order[at], -1))
    return table.contiguous(), len(order)


def _rows(lens, page, table):
    """Cache row of position s of sequence b as a padded [B, Lmax] tensor (0 past a length)."""
    L = torch.tensor(lens, device=DEV)
    s = torch.arange(max(max(lens), 1), device=DEV)
    if page:
        r = table.long()[:, (s // page).clamp(max=table.shape[1] - 1)] * page + s % page
    else:
        r = (torch.cumsum(L, 0) - L)[:, None] + s[None]
    return torch.where(s[None] < L[:, None], r, torch.zeros_like(r))


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    st = {"case": case}
    op = case["op"]
    if op == "norm":
        dt, rows, d = _DT[case["dtype"]], case["rows"], case["d"]
        x = _randn(g, (rows, max(d, case["stride"])), dt)
        off = 8 if case["stride"] >= d + 8 else 0
        st["x"] = x[:, off:off + d]
        st["w"] = (1 + 0.1 * torch.randn(d, generator=g, device=DEV)).to(dt)
        st["residual"] = _randn(g, (rows, d), dt, 2.0) if case["residual"] else None
        return st
    q_lens, k_lens = _lens(case)
    D, page = case["d_c"] + case["d_rope"], case["page"]
    dt = _DT[case.get("dtype", "bf16")]
    B = case["B"]
    st.update(q_lens=q_lens, k_lens=k_lens, cu_q=_offsets(q_lens), cu_k=_offsets(k_lens),
              table=None, num_pages=0, scale=D ** -0.5)
    P = case.get("prefix", 0)
    if page:
        lens = k_lens + [P] if op == "prefix" else k_lens
        table, st["num_pages"] = _pages(lens, page, g)
        if op == "prefix":
            st["prefix_table"] = table[B, :max(1, -(-P // page))].contiguous()
            table = table[:B]
        st["table"] = table.contiguous()
        total = st["num_pages"] * page
    else:
        total = sum(k_lens)
    st["rows"] = _rows(k_lens, page, st["table"])
    st["kv"] = _randn(g, (total, D), dt)
    if op == "evict":
        n = [min(L, case["budget"]) for L in k_lens]
        st["acc"] = torch.rand(B, max(k_lens), generator=g, device=DEV).pow_(6) * 8
        st["k_idx"] = _randn(g, (total, 128), torch.float8_e4m3fn).view(torch.uint8)
        st["k_scale"] = torch.rand(total, generator=g, device=DEV) + 0.5
        st["n"] = torch.tensor(n, device=DEV)
        st["table_out"], rows_out = None, sum(n)
        if page:
            st["table_out"], pages_out = _pages(n, page, g)
            rows_out = pages_out * page
        st["rows_out"] = _rows(n, page, st["table_out"])
        st["kv_out"] = torch.zeros(rows_out, D, dtype=dt, device=DEV)
        st["k_idx_out"] = torch.zeros(rows_out, 128, dtype=torch.uint8, device=DEV)
        st["k_scale_out"] = torch.zeros(rows_out, device=DEV)
    else:
        TQ, H = sum(q_lens), case["heads"]
        st["q"] = _randn(g, (TQ, H, D), dt)
        T = torch.tensor(q_lens, device=DEV)
        L = torch.tensor(k_lens, device=DEV)
        st["seq"] = torch.repeat_interleave(torch.arange(B, device=DEV), T)
        st["row_in"] = torch.arange(TQ, device=DEV) - (torch.cumsum(T, 0) - T)[st["seq"]]
        st["pos"] = (L - T)[st["seq"]] + st["row_in"]
    if op == "prefix":
        if page:
            s = torch.arange(P, device=DEV)
            st["prefix_rows"] = st["prefix_table"].long()[s // page] * page + s % page
            st["prefix_kv"] = None
        else:
            st["prefix_kv"] = _randn(g, (P, D), dt)
    if op == "weights":
        k = case["top_k"]
        Lm = max(k_lens)
        r = torch.rand(TQ, Lm, generator=g, device=DEV)
        r.masked_fill_(torch.arange(Lm, device=DEV)[None] > st["pos"][:, None], -1.0)
        kk = min(k, Lm)
        v, i = r.topk(kk, dim=1)
        i = torch.where(v >= 0, i, torch.full_like(i, 1 << 30)).sort(dim=1).values
        idx = torch.full((TQ, k), -1, dtype=torch.int32, device=DEV)
        idx[:, :kk] = torch.where(i < (1 << 30), i, torch.full_like(i, -1)).to(torch.int32)
        st["idx"] = idx
        S = _selected_logits(st, torch.float32)
        st["lse"] = torch.logsumexp(S, dim=2).contiguous()
        st["acc"] = torch.rand(B, Lm, generator=g, device=DEV)
    if own:
        st["P"] = _problem(st)
    return st


def _problem(st):
    import sparse_attention_lightning_gb300 as dsa
    c = st["case"]
    dt = c.get("dtype", "bf16")
    return dsa.Problem(st["cu_q"], st["cu_k"], q_lens=st["q_lens"], k_lens=st["k_lens"], h_idx=64,
                       d_idx=128, h=c.get("heads", 128), d_c=c["d_c"], d_rope=c["d_rope"],
                       top_k=c.get("top_k", 2048), idx_dtype="e4m3", kv_dtype=dt, out_dtype=dt,
                       block_table=st["table"], page_size=c["page"], num_pages=st["num_pages"])


# ---------------------------------------------------------------------------
# One pass.

def run(st):
    op = st["case"]["op"]
    if own:
        return _OWN[op](st)
    return _PLAIN[op](st)


def _own_norm(st):
    import sparse_attention_lightning_gb300 as dsa
    quant = st["case"]["quant"]
    y, h, codes, scale = dsa.add_rmsnorm(st["x"], st["w"], residual=st["residual"], eps=1e-6,
                                         quant=None if quant == "none" else quant)
    return _norm_outputs(y, h, codes, scale)


def _norm_outputs(y, h, codes, scale):
    out = {} if h is None else {"h": h}
    if codes is None:
        out["y"] = y
        return out
    out["codes"] = codes.view(torch.float8_e4m3fn)
    out["scale"] = scale if scale.dtype == torch.float32 else scale.view(torch.float8_e8m0fnu)
    return out


def _plain_norm(st):
    x, w, res, quant = st["x"], st["w"].float(), st["residual"], st["case"]["quant"]
    h = x.float()
    if res is not None:
        h = h + res.float()
    y = h * torch.rsqrt((h * h).mean(dim=1, keepdim=True) + 1e-6) * w
    h = None if res is None else h.to(x.dtype)
    if quant == "none":
        return _norm_outputs(y.to(x.dtype), h, None, None)
    if quant == "e4m3":  # one fp32 scale a row
        scale = y.abs().amax(dim=1) / 448.0
        scale = torch.where(scale < 2.0 ** -126, torch.ones_like(scale), scale)
        codes = (y / scale[:, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
        return _norm_outputs(None, h, codes.view(torch.uint8), scale)
    # the smallest power of two 2^e with amax <= 448 * 2^e for 32 elements
    yg = y.reshape(y.shape[0], -1, 32)
    amax = yg.abs().amax(dim=2)
    m, e = torch.frexp(amax)
    e = e - 9 + (m > 0.875).to(e.dtype)
    e = torch.where(amax > 0, e, torch.zeros_like(e)).clamp(-127, 127)
    codes = (yg * torch.exp2(-e.float())[:, :, None]).clamp(-448.0, 448.0)
    return _norm_outputs(None, h, codes.to(torch.float8_e4m3fn).view(torch.uint8).reshape(y.shape),
                         (e + 127).to(torch.uint8))


def _own_prefix(st):
    import sparse_attention_lightning_gb300 as dsa
    c = st["case"]
    if c["page"]:
        out, lse = dsa.prefix_mla_attn(st["P"], st["q"], st["kv"],
                                       prefix_table=st["prefix_table"], prefix_len=c["prefix"])
    else:
        out, lse = dsa.prefix_mla_attn(st["P"], st["q"], st["kv"], prefix_kv=st["prefix_kv"])
    return {"out": out, "lse": lse}


def _plain_prefix(st):
    c, q = st["case"], st["q"].float()
    TQ, H, D = q.shape
    B, Tm, dc = c["B"], max(st["q_lens"]), c["d_c"]
    pre = (st["kv"][st["prefix_rows"]] if c["page"] else st["prefix_kv"]).float()
    suf = st["kv"][st["rows"]].float()                                    # [B, Lm, D]
    S1 = torch.matmul(q.reshape(TQ * H, D), pre.T).reshape(TQ, H, -1) * st["scale"]
    qp = q.new_zeros(B, Tm, H, D)
    qp[st["seq"], st["row_in"]] = q
    S2 = torch.matmul(qp.reshape(B, Tm * H, D), suf.transpose(1, 2)).reshape(B, Tm, H, -1)
    S2 = S2[st["seq"], st["row_in"]] * st["scale"]                        # [TQ, H, Lm]
    hidden = torch.arange(suf.shape[1], device=DEV)[None] > st["pos"][:, None]
    S2 = S2.masked_fill(hidden[:, None], -math.inf)
    m = S2.amax(dim=2, keepdim=True)
    if S1.shape[2]:
        m = torch.maximum(m, S1.amax(dim=2, keepdim=True))
    p1, p2 = torch.exp(S1 - m), torch.exp(S2 - m)
    l = p1.sum(dim=2, keepdim=True) + p2.sum(dim=2, keepdim=True)
    pp = q.new_zeros(B, Tm, H, p2.shape[2])
    pp[st["seq"], st["row_in"]] = p2
    o2 = torch.matmul(pp.reshape(B, Tm * H, -1), suf[:, :, :dc]).reshape(B, Tm, H, dc)
    o = torch.matmul(p1.reshape(TQ * H, -1), pre[:, :dc]).reshape(TQ, H, dc)
    o = (o + o2[st["seq"], st["row_in"]]) / l
    return {"out": o.to(st["q"].dtype), "lse": (m + torch.log(l))[:, :, 0]}


def _selected_logits(st, dtype):
    """scale * q . kv of the selected positions, -inf in the padding: [TQ, H, k]."""
    idx = st["idx"].long()
    rows = st["rows"][st["seq"][:, None], idx.clamp(min=0)]
    S = torch.matmul(st["q"].to(dtype), st["kv"][rows].to(dtype).transpose(1, 2)) * st["scale"]
    return S.masked_fill((idx < 0)[:, None], -math.inf)


def _own_weights(st):
    import sparse_attention_lightning_gb300 as dsa
    return {"acc": dsa.accumulate_attn_weights(st["P"], st["q"], st["kv"], st["idx"], st["lse"],
                                               st["acc"])}


def _plain_weights(st):
    p = torch.exp(_selected_logits(st, torch.float32) - st["lse"][:, :, None]).sum(dim=1)
    acc = st["acc"]
    at = st["seq"][:, None] * acc.shape[1] + st["idx"].long().clamp(min=0)
    total = acc.double().reshape(-1)  # long sums of many queries
    total.index_add_(0, at.reshape(-1), p.double().reshape(-1))
    acc.copy_(total.reshape(acc.shape))
    return {"acc": acc}


def _own_evict(st):
    import sparse_attention_lightning_gb300 as dsa
    c = st["case"]
    r = dsa.evict(st["P"], st["acc"], c["budget"], sink=c["sink"], recent=c["recent"],
                  kv=st["kv"], k_idx=st["k_idx"], k_scale=st["k_scale"], kv_out=st["kv_out"],
                  k_idx_out=st["k_idx_out"], k_scale_out=st["k_scale_out"],
                  block_table_out=st["table_out"])
    return _evict_outputs(st, r.kept, r.cu_k, r.acc)


def _evict_outputs(st, kept, cu_k, acc):
    return {"kept": kept, "cu_k": cu_k, "acc": acc, "kv": st["kv_out"],
            "k_idx": st["k_idx_out"].view(torch.float8_e4m3fn), "k_scale": st["k_scale_out"]}


def _plain_evict(st):
    c, acc, n = st["case"], st["acc"], st["n"]
    B, Lm = acc.shape
    budget = c["budget"]
    s = torch.arange(Lm, device=DEV)[None]
    L = (st["cu_k"][1:] - st["cu_k"][:-1]).long()[:, None]
    key = torch.where((s < c["sink"]) | (s >= L - c["recent"]), math.inf, acc)
    key = torch.where(s < L, key, -math.inf)
    order = torch.sort(key, dim=1, descending=True, stable=True).indices
    chosen = torch.zeros(B, Lm, dtype=torch.bool, device=DEV)
    chosen.scatter_(1, order, s.expand(B, Lm) < n[:, None])
    slot = torch.cumsum(chosen, dim=1) - 1
    b, pos = chosen.nonzero(as_tuple=True)
    to = slot[b, pos]
    kept = torch.full((B, budget), -1, dtype=torch.int32, device=DEV)
    kept[b, to] = pos.to(torch.int32)
    acc_out = acc.new_zeros(B, budget)
    acc_out[b, to] = acc[b, pos]
    src, dst = st["rows"][b, pos], st["rows_out"][b, to]
    st["kv_out"][dst] = st["kv"][src]
    st["k_idx_out"][dst] = st["k_idx"][src]
    st["k_scale_out"][dst] = st["k_scale"][src]
    cu = torch.zeros(B + 1, dtype=torch.int32, device=DEV)
    cu[1:] = torch.cumsum(n, 0)
    return _evict_outputs(st, kept, cu, acc_out)


_OWN = {"norm": _own_norm, "prefix": _own_prefix, "weights": _own_weights, "evict": _own_evict}
_PLAIN = {"norm": _plain_norm, "prefix": _plain_prefix, "weights": _plain_weights,
          "evict": _plain_evict}


# ---------------------------------------------------------------------------
# The definitions in 64 bits, one sequence or one block of rows at a time.

def exact(case, seed):
    st = prepare(case, seed)
    return {"norm": _exact_norm, "prefix": _exact_prefix, "weights": _exact_weights,
            "evict": _exact_evict}[case["op"]](st)


def _e4m3(v):
    """The E4M3 values next to v: 3 bits behind the leading one, exponents from -6, at most 448."""
    v = v.clamp(-448.0, 448.0)
    ex = torch.frexp(v)[1].clamp(min=-5) - 1
    step = torch.ldexp(torch.ones_like(v), ex - 3)
    return torch.round(v / step) * step


def _exact_norm(st):
    c = st["case"]
    h = st["x"].double()
    out = {}
    if st["residual"] is not None:
        h = h + st["residual"].double()
        out["h"] = h
    y = h / torch.sqrt(h.square().sum(dim=1, keepdim=True) / c["d"] + 1e-6) * st["w"].double()
    if c["quant"] == "none":
        out["y"] = y
    elif c["quant"] == "e4m3":
        out["scale"] = y.abs().max(dim=1).values / 448
        out["codes"] = _e4m3(y / out["scale"][:, None])
    else:
        g = y.reshape(-1, 32)
        two = torch.exp2(torch.ceil(torch.log2(g.abs().max(dim=1).values / 448)))
        out["codes"] = _e4m3(g / two[:, None]).reshape(y.shape)
        out["scale"] = two.reshape(c["rows"], -1)
    return out


def _exact_prefix(st):
    c = st["case"]
    kv = st["kv"]
    pre = (kv[st["prefix_rows"]] if c["page"] else st["prefix_kv"]).double()
    outs, lses, t0 = [], [], 0
    for b, (T, L) in enumerate(zip(st["q_lens"], st["k_lens"])):
        keys = torch.cat((pre, kv[st["rows"][b, :L]].double()))
        for i in range(T):
            k = keys[:c["prefix"] + L - T + i + 1]
            S = (st["q"][t0 + i].double() @ k.T) * st["scale"]
            lse = torch.logsumexp(S, dim=1)
            outs.append(torch.exp(S - lse[:, None]) @ k[:, :c["d_c"]])
            lses.append(lse)
        t0 += T
    return {"out": torch.stack(outs), "lse": torch.stack(lses)}


def _exact_weights(st):
    acc = st["acc"].double()
    seq = st["seq"].tolist()
    for t in range(len(seq)):
        i = st["idx"][t]
        i = i[i >= 0].long()
        k = st["kv"][st["rows"][seq[t], i]].double()
        S = (st["q"][t].double() @ k.T) * st["scale"]
        acc[seq[t], i] += torch.exp(S - st["lse"][t].double()[:, None]).sum(dim=0)
    return {"acc": acc}


def _exact_evict(st):
    c = st["case"]
    B, budget = c["B"], c["budget"]
    kept = torch.full((B, budget), -1, dtype=torch.int32, device=DEV)
    acc = torch.zeros(B, budget, dtype=torch.float64, device=DEV)
    kv, ki, ks = (torch.zeros(st[n].shape, dtype=torch.float64, device=DEV)
                  for n in ("kv_out", "k_idx_out", "k_scale_out"))
    cu = [0]
    for b, L in enumerate(st["k_lens"]):
        a = st["acc"][b, :L].tolist()
        n = min(L, budget)
        must = [s for s in range(L) if s < c["sink"] or s >= L - c["recent"]]
        if L <= budget:
            pick = list(range(L))
        else:
            free = sorted((s for s in range(c["sink"], L - c["recent"])), key=lambda s: (-a[s], s))
            pick = sorted(must + free[:n - len(must)])
        p = torch.tensor(pick, device=DEV)
        kept[b, :n] = p.to(torch.int32)
        acc[b, :n] = st["acc"][b, p].double()
        src, dst = st["rows"][b, p], st["rows_out"][b, :n]
        kv[dst] = st["kv"][src].double()
        ki[dst] = st["k_idx"][src].view(torch.float8_e4m3fn).double()
        ks[dst] = st["k_scale"][src].double()
        cu.append(cu[-1] + n)
    return {"kept": kept, "cu_k": torch.tensor(cu, dtype=torch.int32, device=DEV), "acc": acc,
            "kv": kv, "k_idx": ki, "k_scale": ks}
