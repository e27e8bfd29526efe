"""What the operators of the 4-bit latent cache cost: rotary positions with several axes, rows written to
and read from the cache, sparse MLA attention over it, and the pages that hold a cache (forked, reserved,
freed, compacted).

`run` computes an operator in elementary torch operations (own = False) or through the
framework's calls (own = True), on the same state.
"""
import math
import random

import torch

own = False


# ---------------------------------------------------------------------------
# Cases.

def listed():
    return [
        # the query of one decoded token, all heads: latency only
        dict(name="rotate, one token", op="rotate", T=1, heads=128, d=576, d_rope=64, axes=3,
             interleaved=True, dtype="bf16", inverse=False),
        # the queries of an 8k prefill with image and video positions, rope columns of [8192, 128, 576] in place
        dict(name="rotate, 8k prefill", op="rotate", T=8192, heads=128, d=576, d_rope=64, axes=3,
             interleaved=True, dtype="bf16", inverse=False),
        # a few short fp32 sequences of the tiny workload's widths get one or more tokens, and are read back
        dict(name="kv4, tiny fp32", op="kv4", B=5, d_c=64, d_rope=16, t_max=3, l_max=61, page=16,
             dtype="f32", lens_seed=1),
        # an 8k prompt's latent rows go to the cache and come back for dense attention
        dict(name="kv4, 8k prompt", op="kv4", B=1, d_c=512, d_rope=64, t_max=8192, l_max=8192, page=0,
             dtype="bf16", lens_seed=1),
        # one decode step of the 32-sequence workload
        dict(name="attn, decode", op="attn", B=32, heads=128, d_c=512, d_rope=64, t_max=1, l_min=8192,
             l_max=32768, top_k=2048, page=0, dtype="bf16", lens_seed=3),
        # decode of 128 sequences with 128k positions each: byte offsets past 32 bits
        dict(name="attn, 128 x 128k", op="attn", B=128, heads=128, d_c=512, d_rope=64, t_max=1,
             l_min=131072, l_max=131072, top_k=2048, page=64, dtype="bf16", lens_seed=4),
        # speculative steps of a few sequences with 16 heads a GPU, odd lengths, paged
        dict(name="attn, 16 heads", op="attn", B=13, heads=16, d_c=512, d_rope=64, t_max=4, l_min=900,
             l_max=5001, top_k=999, page=64, dtype="bf16", lens_seed=5),
        # a prefill chunk of 1024 queries behind 7k positions
        dict(name="attn, prefill chunk", op="attn", B=1, heads=128, d_c=512, d_rope=64, t_max=1024,
             l_min=8192, l_max=8192, top_k=2048, page=0, dtype="bf16", lens_seed=1),
        # four samples of each of three prompts start over: their pages freed, the prompts forked, room for new tokens
        dict(name="pages, 3 x 4 samples", op="pages", parents=3, per=4, l_max=700, grow=1, page=64,
             spare=40, lens_seed=7),
        # sixteen samples of each of 32 prompts of up to 32k, room for 256 new tokens
        dict(name="pages, 32 x 16 samples", op="pages", parents=32, per=16, l_max=32768, grow=256,
             page=64, spare=500, lens_seed=8),
        # a small pool after a few sequences have left
        dict(name="compact, small", op="compact", B=9, l_max=500, gone=4, page=16, lens_seed=9),
        # a pool of a million rows, half of whose sequences have left
        dict(name="compact, 1M rows", op="compact", B=64, l_max=32768, gone=32, page=64, lens_seed=10),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(("rotate", "kv4", "attn", "attn", "pages", "compact"))
    seed = rng.randint(1, 1 << 20)
    page = rng.choice((0, 16, 64, 256))
    if op == "rotate":
        T, heads = _log(rng, 1, 8192), rng.choice((1, 1, 8, 16, 20, 64, 128))
        d_rope = rng.choice((64, 64, 64, 16, 32, 48, 128, 256))
        return dict(op=op, T=max(1, min(T, 8192 * 128 * 64 // (heads * d_rope))), heads=heads,
                    d=d_rope + rng.choice((0, 64, 512)), d_rope=d_rope, axes=rng.choice((1, 2, 3, 3, 4)),
                    interleaved=rng.random() < 0.6, dtype=rng.choice(("bf16", "bf16", "f32")),
                    inverse=rng.random() < 0.2)
    f32 = rng.random() < 0.15
    if op == "kv4":
        d_c, d_rope = rng.choice(((512, 64), (512, 64), (64, 16), (256, 32), (128, 64), (512, 0), (1024, 64), (16, 0)))
        B = _log(rng, 1, 64)
        t_max = _log(rng, 1, max(1, 8192 // B))
        return dict(op=op, B=B, d_c=d_c, d_rope=d_rope, t_max=t_max,
                    l_max=max(t_max, min(8192 // B, _log(rng, 1, 8192))), page=page,
                    dtype="f32" if f32 else "bf16", lens_seed=seed)
    if op == "attn":
        d_c, d_rope = (64, 16) if f32 else (512, 64) if rng.random() < 0.8 else rng.choice(((256, 32), (64, 16)))
        B = _log(rng, 1, 64)
        t_max = rng.choice((1, 1, 1, 2, 5, rng.randint(6, 40)))
        l_max = max(t_max, _log(rng, 10, 32768))
        top_k = min(_log(rng, 1, 2048), 131072 // (B * t_max))
        heads = rng.choice((1, 8, 16, 20, 64, 128))
        if d_c != 512:
            top_k = min(top_k, max(1, (1 << 22) // (B * t_max * heads)))
        return dict(op=op, B=B, heads=heads, d_c=d_c, d_rope=d_rope, t_max=t_max,
                    l_min=max(t_max, l_max // 4), l_max=l_max, top_k=max(1, top_k), page=page,
                    dtype="f32" if f32 else "bf16", lens_seed=seed)
    page = page or 32
    if op == "pages":
        parents, per = _log(rng, 1, 32), _log(rng, 1, 16)
        return dict(op=op, parents=parents, per=per, l_max=_log(rng, 1, 32768), grow=_log(rng, 1, 256), page=page,
                    spare=rng.randint(0, 500), lens_seed=seed)
    B = _log(rng, 1, 64)
    return dict(op=op, B=B, l_max=_log(rng, 1, 32768), gone=rng.randint(0, B), page=page, lens_seed=seed)


def _lens(case):
    """(new tokens, lengths) of a case's sequences, from the case alone."""
    r = random.Random(case["lens_seed"])
    op, n = case["op"], case["parents"] if case["op"] == "pages" else case["B"]
    if op in ("pages", "compact"):
        lo = max(1, case["l_max"] // 4)
        return None, [r.randint(lo, case["l_max"]) for _ in range(n)]
    T = case["t_max"]
    q = [T if r.random() < 0.5 else r.randint(1, T) for _ in range(n)]
    lo = case.get("l_min", 1)
    return q, [r.randint(max(t, lo), max(t, case["l_max"])) for t in q]


def _row_bytes(case):
    """Bytes of a row of the 4-bit cache: codes, rope columns in bf16, a scale for 16 columns, whole 16 bytes."""
    return -(-(case["d_c"] // 2 + case["d_c"] // 16 + 2 * case["d_rope"]) // 16) * 16


# the caches that share the pages: a 4-bit latent row, an FP8 index key and its scale
_CACHES = (("kv4", 416, torch.uint8), ("k_idx", 128, torch.uint8), ("k_scale", None, torch.float32))
_CACHE_ROW = 416 + 128 + 4


def _pairs(case):
    q, k = _lens(case)
    return sum(min(case["top_k"], L - t + i + 1) for t, L in zip(q, k) for i in range(t))


def work(case):
    op = case["op"]
    b = 2 if case.get("dtype") == "bf16" else 4
    if op == "rotate":
        n = case["T"] * case["heads"] * case["d_rope"]
        return {"bytes": 2 * b * n + 4 * case["axes"] * case["T"], "flops": 3 * n}
    if op == "kv4":
        q, k = _lens(case)
        D, rb = case["d_c"] + case["d_rope"], _row_bytes(case)
        return {"bytes": sum(q) * (b * D + rb) + sum(k) * (rb + b * D), "flops": 4 * D * (sum(q) + sum(k))}
    if op == "attn":
        q, k = _lens(case)
        n, D, H, TQ = _pairs(case), case["d_c"] + case["d_rope"], case["heads"], sum(q)
        return {"bytes": min(n, sum(k)) * _row_bytes(case) + 4 * TQ * case["top_k"] + TQ * H * (b * (D + case["d_c"]) + 4),
                "flops": 2 * H * (D + case["d_c"]) * n}
    _, k = _lens(case)
    page = case["page"]
    if op == "pages":
        held = sum(-(-L // page) + -(-(L + case["grow"]) // page) for L in k)
        rows = sum(L % page for L in k)
        return {"bytes": case["per"] * (2 * rows * _CACHE_ROW + 2 * 8 * held) + 8 * len(k), "flops": 0}
    moved, live = _moved(case)
    return {"bytes": 2 * moved * page * _CACHE_ROW + 8 * live + 8 * moved, "flops": 0}


def _moved(case):
    """(about the pages that move, the live pages): live ones are anywhere in the pool."""
    _, k = _lens(case)
    need = [-(-L // case["page"]) for L in k]
    live, every = sum(need[case["gone"]:]), sum(need) + 3
    return int(live * (1 - live / every)), live


# ---------------------------------------------------------------------------
# Inputs.

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
DEV = "cuda"


def _randn(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _offsets(lens):
    c = [0]
    for n in lens:
        c.append(c[-1] + n)
    return _i32(c)


def _table(need, order, width):
    """Table rows [len(need), width] that take pages from `order` in turn, -1 behind them."""
    per = torch.tensor(need, device=DEV)
    first = torch.cumsum(per, 0) - per
    slot = torch.arange(width, device=DEV)
    at = (first[:, None] + slot[None]).clamp(max=len(order) - 1)
    return torch.where(slot[None] < per[:, None], order[at], torch.full_like(order[at], -1)).contiguous()


def _rows(lens, page, table):
    """Cache row of position s of sequence b as a padded [B, Lmax] tensor (0 past a length)."""
    L = torch.tensor(lens, device=DEV)
    s = torch.arange(max(max(lens), 1), device=DEV)
    if page:
        r = table.long()[:, (s // page).clamp(max=table.shape[1] - 1)] * page + s % page
    else:
        r = (torch.cumsum(L, 0) - L)[:, None] + s[None]
    return torch.where(s[None] < L[:, None], r, torch.zeros_like(r))


def _sections(case):
    """Pairs of each axis: the first axis a half, the others equal parts of the rest."""
    n, a = case["d_rope"] // 2, case["axes"]
    rest = n // 2 // max(1, a - 1) if a > 1 else 0
    return [n - rest * (a - 1)] + [rest] * (a - 1)


def _random_cache(g, rows, case):
    """Rows of a 4-bit cache with values of order one."""
    d_c, d_rope, rb = case["d_c"], case["d_rope"], _row_bytes(case)
    kv4 = torch.randint(0, 256, (rows, rb), generator=g, device=DEV, dtype=torch.uint8)
    at = d_c // 2
    if d_rope:
        kv4[:, at:at + 2 * d_rope] = _randn(g, (rows, d_rope), torch.bfloat16).view(torch.uint8)
        at += 2 * d_rope
    kv4[:, at:at + d_c // 16] = torch.randint(0x62, 0x70, (rows, d_c // 16), generator=g, device=DEV, dtype=torch.uint8)
    kv4[:, at + d_c // 16:] = 0
    return kv4


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    st = {"case": case}
    op = case["op"]
    if op == "rotate":
        st["x"] = _randn(g, (case["T"], case["heads"], case["d"]), _DT[case["dtype"]])
        # times and rows of long videos: positions far from zero
        st["pos"] = torch.randint(0, 1 << 20, (case["axes"], case["T"]), generator=g, device=DEV, dtype=torch.int32)
        n = case["d_rope"] // 2
        st["freq"] = [10000.0 ** (-i / n) for i in range(n)]
        st["axis"] = [a for a, k in enumerate(_sections(case)) for _ in range(k)]
        st["turn"] = torch.tensor(st["freq"], dtype=torch.float64, device=DEV)
        st["axis_of"] = torch.tensor(st["axis"], device=DEV)
        if own:
            import sparse_attention_lightning_gb300 as dsa
            st["rotary"] = dsa.Rotary(case["d_rope"], sections=_sections(case), inv_freq=st["freq"],
                                      interleaved=case["interleaved"])
        return st
    q_lens, k_lens = _lens(case)
    page = case["page"]
    if op in ("pages", "compact"):
        return _prepare_pages(case, st, g, k_lens)
    d_c, d_rope, dt = case["d_c"], case["d_rope"], _DT[case["dtype"]]
    D, TQ = d_c + d_rope, sum(q_lens)
    st.update(q_lens=q_lens, k_lens=k_lens, cu_q=_offsets(q_lens), cu_k=_offsets(k_lens), table=None,
              num_pages=0, scale=D ** -0.5)
    if page:
        need = [-(-n // page) for n in k_lens]
        st["num_pages"] = sum(need) + 3
        order = torch.randperm(st["num_pages"], generator=g, device=DEV).to(torch.int32)
        st["table"] = _table(need, order, max(need))
    total = st["num_pages"] * page if page else sum(k_lens)
    st["rows"] = _rows(k_lens, page, st["table"])
    T, L = torch.tensor(q_lens, device=DEV), torch.tensor(k_lens, device=DEV)
    st["seq"] = torch.repeat_interleave(torch.arange(len(q_lens), device=DEV), T)
    st["pos"] = (L - T)[st["seq"]] + torch.arange(TQ, device=DEV) - (torch.cumsum(T, 0) - T)[st["seq"]]
    st["kv4"] = _random_cache(g, total, case)
    if op == "kv4":
        wide = _randn(g, (TQ, D + 8), dt)  # a slice of a wider projection
        st["latent"], st["k_rope"] = wide[:, :d_c], wide[:, d_c:D]
        st["packed"] = torch.cat([st["rows"][b, :n] for b, n in enumerate(k_lens)])
    else:
        st["q"] = _randn(g, (TQ, case["heads"], D), dt)
        k, Lm = case["top_k"], max(k_lens)
        r = torch.rand(TQ, Lm, generator=g, device=DEV)
        r.masked_fill_(torch.arange(Lm, device=DEV)[None] > st["pos"][:, None], -1.0)
        kk = min(k, Lm)
        v, i = r.topk(kk, dim=1)
        i = torch.where(v >= 0, i, torch.full_like(i, 1 << 30)).sort(dim=1).values
        st["idx"] = torch.full((TQ, k), -1, dtype=torch.int32, device=DEV)
        st["idx"][:, :kk] = torch.where(i < (1 << 30), i, torch.full_like(i, -1)).to(torch.int32)
    if own:
        import sparse_attention_lightning_gb300 as dsa
        st["P"] = dsa.Problem(st["cu_q"], st["cu_k"], q_lens=q_lens, k_lens=k_lens, h_idx=64, d_idx=128,
                              h=case.get("heads", 128), d_c=d_c, d_rope=d_rope, top_k=case.get("top_k", 2048),
                              idx_dtype="e4m3", kv_dtype=case["dtype"], out_dtype=case["dtype"],
                              block_table=st["table"], page_size=page, num_pages=st["num_pages"])
    return st


def _caches(g, pages, page):
    rows = pages * page
    return {name: torch.randint(0, 256, (rows, w), generator=g, device=DEV, dtype=dt) if w else
            torch.rand(rows, generator=g, device=DEV) for name, w, dt in _CACHES}


def _prepare_pages(case, st, g, k_lens):
    page = case["page"]
    need = [-(-n // page) for n in k_lens]
    if case["op"] == "compact":
        pages = sum(need) + 3
        order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
        table = _table(need, order, max(need))
        table[:case["gone"]] = -1
        refs = torch.zeros(pages, dtype=torch.int32, device=DEV)
        refs.index_add_(0, table.clamp(min=0).reshape(-1), (table >= 0).to(torch.int32).reshape(-1))
        st.update(table0=table, refs0=refs, table=table.clone(), refs=refs.clone(), pages=pages)
        st["caches"] = _caches(g, pages, page)
        return st
    n, per, grow = len(k_lens), case["per"], case["grow"]
    width = max(-(-(L + grow) // page) for L in k_lens)
    kids = [p for p in range(n) for _ in range(per)]
    own_pages = [-(-(k_lens[p] + grow) // page) - k_lens[p] // page for p in kids]
    pages = sum(need) + sum(own_pages) + case["spare"]
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table = torch.full((n + len(kids), width), -1, dtype=torch.int32, device=DEV)
    table[:n] = _table(need, order, width)
    # the samples of the step before: the prompt's whole pages, then pages of their own
    mine = _table(own_pages, order[sum(need):], width + 1)
    j = torch.arange(width, device=DEV)[None]
    full = torch.tensor([k_lens[p] // page for p in kids], device=DEV)[:, None]
    own_at = torch.gather(mine, 1, (j - full).clamp(0, width))
    table[n:] = torch.where(j < full, table[:n][torch.tensor(kids, device=DEV)], own_at)
    refs = torch.zeros(pages, dtype=torch.int32, device=DEV)
    refs.index_add_(0, table.clamp(min=0).reshape(-1), (table >= 0).to(torch.int32).reshape(-1))
    st.update(table=table, refs=refs, pages=pages, src=_i32(kids), dst=_i32(list(range(n, n + len(kids)))),
              lens=_i32([k_lens[p] for p in kids]), new_lens=_i32([k_lens[p] + grow for p in kids]))
    st["caches"] = _caches(g, pages, page)
    return st


# ---------------------------------------------------------------------------
# One pass.

def run(st):
    op = st["case"]["op"]
    if own:
        return _OWN[op](st)
    return _PLAIN[op](st)


def _own_rotate(st):
    import sparse_attention_lightning_gb300 as dsa
    c = st["case"]
    x = st["x"][..., c["d"] - c["d_rope"]:]
    return {"x": dsa.rotate_axes(x, st["pos"], st["rotary"], out=x, inverse=c["inverse"])}


def _plain_rotate(st):
    c = st["case"]
    d = c["d_rope"]
    x = st["x"][..., c["d"] - d:]
    angle = st["pos"].double()[st["axis_of"]].T * st["turn"]  # [T, pairs]
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    if c["inverse"]:
        sin = -sin
    f = x.float()
    a, b = (f[..., 0::2], f[..., 1::2]) if c["interleaved"] else (f[..., :d // 2], f[..., d // 2:])
    u, v = a * cos - b * sin, a * sin + b * cos
    y = torch.stack((u, v), dim=-1).flatten(-2) if c["interleaved"] else torch.cat((u, v), dim=-1)
    x.copy_(y)
    return {"x": x}


def _own_kv4(st):
    import sparse_attention_lightning_gb300 as dsa
    dsa.write_kv4(st["P"], st["latent"], st["k_rope"], st["kv4"])
    return {"kv": dsa.read_kv4(st["P"], st["kv4"])}


# Bits of the codes' 32-bit words: element 2k of eight at bit 4k, element 2k + 1 at bit 16 + 4k.
_SHIFT = [4 * (e // 2) + 16 * (e % 2) for e in range(8)]


def _decode(rows, case, dtype):
    """Rows of the cache [..., row bytes] as [..., d_c + d_rope]."""
    d_c, d_rope = case["d_c"], case["d_rope"]
    at = d_c // 2 + 2 * d_rope
    words = rows[..., :d_c // 2].contiguous().view(torch.int32)
    shift = torch.tensor(_SHIFT, dtype=torch.int32, device=rows.device)
    code = (words[..., None] >> shift).bitwise_and_(15).flatten(-2)
    value = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=dtype, device=rows.device)
    # a scale byte is an fp16 number without its sign and its seven lowest bits
    scale = (rows[..., at:at + d_c // 16].to(torch.int16) << 7).view(torch.float16).to(dtype)
    lat = value[code].unflatten(-1, (-1, 16)) * scale[..., None]
    rope = rows[..., d_c // 2:at].contiguous().view(torch.bfloat16).to(dtype)
    return torch.cat((lat.flatten(-2), rope), dim=-1)


def _plain_kv4(st):
    c = st["case"]
    d_c = c["d_c"]
    x = st["latent"].float().unflatten(1, (-1, 16))
    raw = (x.abs().amax(dim=2) / 6).clamp(max=61440.0)
    # four significant bits, or steps of 2^-17 below 2^-14: an fp16 number whose seven lowest bits are zero
    step = torch.ldexp(torch.ones_like(raw), (torch.frexp(raw)[1] - 1).clamp(min=-14) - 3)
    scale = torch.round(raw / step) * step
    u = x / torch.where(scale > 0, scale, torch.ones_like(scale))[..., None]
    u = torch.where(scale[..., None] > 0, u, torch.zeros_like(u))
    au = u.abs()
    st2 = torch.where(au < 2, 0.5, torch.where(au < 4, 1.0, 2.0))
    m = (torch.round(au / st2) * st2).clamp(max=6.0)  # 0, .5, 1, 1.5, 2, 3, 4, 6
    code = torch.where(m < 2, 2 * m, torch.where(m < 4, 2 + m, 4 + m / 2)).to(torch.int32)
    code = (code + 8 * (u < 0).to(torch.int32)).flatten(1).unflatten(1, (-1, 8))
    words = (code << torch.tensor(_SHIFT, dtype=torch.int32, device=code.device)).sum(dim=2).to(torch.int32)
    parts = [words.view(torch.uint8)]
    if c["d_rope"]:
        parts.append(st["k_rope"].to(torch.bfloat16).contiguous().view(torch.uint8))
    parts.append((scale.to(torch.float16).view(torch.int16) >> 7).to(torch.uint8))
    row = torch.cat(parts, dim=1)
    kv4 = st["kv4"]
    at = st["rows"][st["seq"], st["pos"]]
    kv4[at] = torch.nn.functional.pad(row, (0, kv4.shape[1] - row.shape[1]))
    return {"kv": _decode(kv4[st["packed"]], c, torch.float32).to(_DT[c["dtype"]])}


def _own_attn(st):
    import sparse_attention_lightning_gb300 as dsa
    out, lse = dsa.sparse_mla_attn4(st["P"], st["q"], st["kv4"], st["idx"])
    return {"out": out, "lse": lse}


def _plain_attn(st):
    c = st["case"]
    idx = st["idx"].long()
    at = st["rows"][st["seq"][:, None], idx.clamp(min=0)]
    if at.numel() < st["kv4"].shape[0]:
        kv = _decode(st["kv4"][at], c, torch.float32)
    else:
        kv = _decode(st["kv4"], c, torch.float32)[at]
    S = torch.matmul(st["q"].float(), kv.transpose(1, 2)) * st["scale"]
    S.masked_fill_((idx < 0)[:, None], -math.inf)
    m = S.amax(dim=2, keepdim=True)
    p = torch.exp(S - m)
    l = p.sum(dim=2, keepdim=True)
    o = torch.matmul(p, kv[..., :c["d_c"]]) / l
    return {"out": o.to(st["q"].dtype), "lse": (m + torch.log(l))[:, :, 0]}


def _own_pages(st):
    import sparse_attention_lightning_gb300 as dsa
    page, table, refs = st["case"]["page"], st["table"], st["refs"]
    caches = list(st["caches"].values())
    dsa.free_pages(table, refs, st["dst"])
    dsa.fork_pages(table, refs, st["src"], st["dst"], st["lens"], page)
    held = dsa.reserve_pages(table, refs, st["dst"], st["lens"], st["new_lens"], page, caches=caches)
    return {"table": table, "refs": refs, "held": held, **st["caches"]}


def _count(refs, pages, by):
    refs.index_add_(0, pages.clamp(min=0).reshape(-1).long(), ((pages >= 0).to(torch.int32) * by).reshape(-1))


def _plain_pages(st):
    page, table, refs = st["case"]["page"], st["table"], st["refs"]
    src, dst, L, N = (st[k].long() for k in ("src", "dst", "lens", "new_lens"))
    j = torch.arange(table.shape[1], device=DEV)[None]
    # free
    _count(refs, table[dst], -1)
    table[dst] = -1
    # fork
    tab = torch.where(j < (-(-L // page))[:, None], table[src], torch.full_like(table[src], -1))
    _count(refs, tab, 1)
    # reserve: the page that the next token goes to is copied where others hold it too, pages behind it are new
    part = (L % page != 0) & (N > L)
    at = (L // page).clamp(max=table.shape[1] - 1)
    old = torch.gather(tab, 1, at[:, None])[:, 0].long().clamp(min=0)
    many = part & (refs[old] > 1)
    n = torch.zeros_like(refs).index_add_(0, old, many.to(torch.int32))
    i = torch.arange(len(L), device=DEV)
    first = torch.full_like(refs, len(L)).scatter_reduce_(0, old, torch.where(many, i, len(L)).to(torch.int32), "amin")
    copy = many & ~((n[old] == refs[old]) & (first[old] == i))
    new = (j >= (-(-L // page))[:, None]) & (j < (-(-N // page))[:, None])
    need = new & ((tab < 0) | (refs[tab.clamp(min=0).long()] > 1)) | ((j == at[:, None]) & copy[:, None])
    free = torch.sort((refs > 0).to(torch.int32), stable=True).indices.to(torch.int32)
    order = torch.cumsum(need.reshape(-1), 0).reshape(need.shape)
    fits = order[:, -1] <= (refs == 0).sum()
    need = need & fits[:, None]
    got = torch.where(need, free[(order - 1).clamp(0, len(free) - 1)], tab)
    _count(refs, torch.where(need, tab, torch.full_like(tab, -1)), -1)
    _count(refs, torch.where(need, got, torch.full_like(tab, -1)), 1)
    table[dst] = got
    # the copied pages' rows
    s = torch.arange(page, device=DEV)[None]
    here = (copy & fits)[:, None] & (s < (L % page)[:, None])
    to = (torch.gather(got, 1, at[:, None]).long() * page + s)[here]
    fro = (old[:, None] * page + s)[here]
    for cache in st["caches"].values():
        cache[to] = cache[fro]
    return {"table": table, "refs": refs, "held": torch.where(fits, N, L).to(torch.int32), **st["caches"]}


def _again(st):
    """The pool as the sequences that left have left it (a pass has compacted it)."""
    st["table"].copy_(st["table0"])
    st["refs"].copy_(st["refs0"])
    return st["table"], st["refs"]


def _own_compact(st):
    import sparse_attention_lightning_gb300 as dsa
    table, refs = _again(st)
    moved, live = dsa.compact_pages(table, refs, st["case"]["page"], caches=list(st["caches"].values()))
    return {"table": table, "refs": refs, "moved": moved, "live": live, **st["caches"]}


def _plain_compact(st):
    table, refs = _again(st)
    page = st["case"]["page"]
    used = refs > 0
    live = used.sum()
    i = torch.arange(len(refs), device=DEV)
    src = (used & (i >= live)).nonzero()[:, 0]
    dst = (~used & (i < live)).nonzero()[:, 0]
    moved = torch.where(used, i, torch.full_like(i, -1))
    moved[src] = dst
    s = torch.arange(page, device=DEV)[None]
    to, fro = (dst[:, None] * page + s).reshape(-1), (src[:, None] * page + s).reshape(-1)
    for cache in st["caches"].values():
        cache[to] = cache[fro]
    table.copy_(torch.where(table >= 0, moved[table.clamp(min=0).long()].to(torch.int32), table))
    refs[dst] = refs[src]
    refs[src] = 0
    return {"table": table, "refs": refs, "moved": moved.to(torch.int32), "live": live.to(torch.int32).reshape(1),
            **st["caches"]}


_OWN = {"rotate": _own_rotate, "kv4": _own_kv4, "attn": _own_attn, "pages": _own_pages, "compact": _own_compact}
_PLAIN = {"rotate": _plain_rotate, "kv4": _plain_kv4, "attn": _plain_attn, "pages": _plain_pages,
          "compact": _plain_compact}


# ---------------------------------------------------------------------------
# The definitions in 64 bits.

def exact(case, seed):
    st = prepare(case, seed)
    return {"rotate": _exact_rotate, "kv4": _exact_kv4, "attn": _exact_attn, "pages": _exact_pages,
            "compact": _exact_compact}[case["op"]](st)


def _exact_rotate(st):
    c = st["case"]
    d = c["d_rope"]
    x = st["x"][..., c["d"] - d:].double()
    y = torch.empty_like(x)
    for i, (f, a) in enumerate(zip(st["freq"], st["axis"])):
        u, v = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + d // 2)
        z = torch.complex(x[..., u], x[..., v])
        turn = st["pos"][a].double() * (-f if c["inverse"] else f)
        z = z * torch.polar(torch.ones_like(turn), turn)[:, None]
        y[..., u], y[..., v] = z.real, z.imag
    return {"x": y}


def _exact_kv4(st):
    """Each latent value as the nearest of the group's multiples, by the points halfway between them."""
    c = st["case"]
    d_c = c["d_c"]
    kv = _exact_rows(st["kv4"], c)
    x = st["latent"].double().reshape(-1, 16)
    amax = x.abs().max(dim=1).values / 6
    sizes = torch.tensor(sorted((m / 8 if e == 0 else 1 + m / 8) * 2.0 ** (max(e, 1) - 15)
                                for e in range(31) for m in range(8)), dtype=torch.float64, device=x.device)
    scale = sizes[_nearest(amax, sizes)][:, None]
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=x.device)
    val = grid[_nearest((x.abs() / scale).nan_to_num(0, posinf=0), grid)] * scale * torch.sign(x)
    at = st["rows"][st["seq"], st["pos"]]
    kv[at] = torch.cat((val.reshape(-1, d_c), st["k_rope"].to(torch.bfloat16).double()), dim=1)
    return {"kv": kv[st["packed"]]}


def _nearest(v, points):
    """Index of the nearest of ascending points; from the middle of two, the one with an even index."""
    mid = (points[1:] + points[:-1]) / 2
    lo, hi = torch.searchsorted(mid, v), torch.searchsorted(mid, v, right=True)
    return torch.where(lo % 2 == 0, lo, hi)


def _exact_rows(rows, c):
    """Decoded cache rows, a byte at a time."""
    d_c, d_rope = c["d_c"], c["d_rope"]
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=rows.device)
    grid = torch.cat((grid, -grid))
    out = torch.empty(rows.shape[0], d_c + d_rope, dtype=torch.float64, device=rows.device)
    b = rows[:, :d_c // 2].long()
    for e in range(8):  # a word's bytes 0, 1 hold its even elements, 2, 3 the odd ones, the lower nibble first
        byte = b[:, (e % 2) * 2 + e // 4::4]
        out[:, e:d_c:8] = grid[byte // 16 if (e // 2) % 2 else byte % 16]
    s = rows[:, d_c // 2 + 2 * d_rope:][:, :d_c // 16].long()
    ex, m = s // 8, (s % 8).double() / 8
    scale = torch.where(ex == 0, m, 1 + m) * torch.exp2(ex.clamp(min=1).double() - 15)
    out[:, :d_c] *= scale.repeat_interleave(16, dim=1)
    if d_rope:
        out[:, d_c:] = rows[:, d_c // 2:d_c // 2 + 2 * d_rope].contiguous().view(torch.bfloat16).double()
    return out


def _exact_attn(st):
    c = st["case"]
    outs, lses = [], []
    seq = st["seq"].tolist()
    for t in range(len(seq)):
        i = st["idx"][t]
        i = i[i >= 0].long()
        k = _exact_rows(st["kv4"][st["rows"][seq[t], i]], c)
        S = (st["q"][t].double() @ k.T) * st["scale"]
        lse = torch.logsumexp(S, dim=1)
        outs.append(torch.exp(S - lse[:, None]) @ k[:, :c["d_c"]])
        lses.append(lse)
    return {"out": torch.stack(outs), "lse": torch.stack(lses)}


def _exact_pages(st):
    page = st["case"]["page"]
    table, refs, scale = st["table"].tolist(), st["refs"].tolist(), st["caches"]["k_scale"].double()
    src, dst, lens, new = (st[k].tolist() for k in ("src", "dst", "lens", "new_lens"))
    for r in dst:
        for p in table[r]:
            refs[p] -= p >= 0
        table[r] = [-1] * len(table[r])
    for s, d, L in zip(src, dst, lens):
        n = -(-L // page)
        table[d] = table[s][:n] + [-1] * (len(table[s]) - n)
        for p in table[d][:n]:
            refs[p] += 1
    before = list(refs)
    free = iter([p for p, n in enumerate(before) if n == 0])
    part = [L % page and before[table[d][L // page]] > 1 and N > L for d, L, N in zip(dst, lens, new)]
    sharers = {}
    for i, (d, L) in enumerate(zip(dst, lens)):
        if part[i]:
            sharers.setdefault(table[d][L // page], []).append(i)
    for i, (d, L, N) in enumerate(zip(dst, lens, new)):
        j = L // page
        if part[i]:
            p = table[d][j]
            if len(sharers[p]) < before[p] or sharers[p][0] != i:
                to, n = next(free), L % page
                scale[to * page:to * page + n] = scale[p * page:p * page + n]
                table[d][j] = to
                refs[p] -= 1
                refs[to] += 1
        for j in range(-(-L // page), -(-N // page)):
            table[d][j] = next(free)
            refs[table[d][j]] += 1
    return {"table": _i32(table), "refs": _i32(refs), "held": _i32(new), "k_scale": scale}


def _exact_compact(st):
    page = st["case"]["page"]
    table, refs, scale = st["table0"].tolist(), st["refs0"].tolist(), st["caches"]["k_scale"].double()
    live = sum(n > 0 for n in refs)
    moved = [p if n > 0 else -1 for p, n in enumerate(refs)]
    holes = iter([p for p in range(live) if refs[p] == 0])
    for p in range(live, len(refs)):
        if refs[p] > 0:
            to = moved[p] = next(holes)
            refs[to], refs[p] = refs[p], 0
            scale[to * page:(to + 1) * page] = scale[p * page:(p + 1) * page]
    table = [[moved[p] if p >= 0 else -1 for p in row] for row in table]
    return {"table": _i32(table), "refs": _i32(refs), "moved": _i32(moved), "live": _i32([live]), "k_scale": scale}
