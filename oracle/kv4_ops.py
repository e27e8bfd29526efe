"""The 4-bit latent cache, rotary positions and pages in fp64 numpy and plain Python, written from their
definitions, one row or one entry at a time.  Nothing is shared with the CUDA path.
"""
from __future__ import annotations

import numpy as np

CODES = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
# scale bytes 0x00 .. 0xf7: an fp16 number's exponent and its three upper mantissa bits
SCALES = np.array([(m / 8 if e == 0 else 1 + m / 8) * 2.0 ** (max(e, 1) - 15) for e in range(31) for m in range(8)])


def row_bytes(d_c, d_rope):
    return -(-(d_c // 2 + 2 * d_rope + d_c // 16) // 16) * 16


def nearest(v, points):
    """Index of the nearest of ascending points, of two as near the one with an even index."""
    mid = (points[1:] + points[:-1]) / 2
    lo, hi = np.searchsorted(mid, v, "left"), np.searchsorted(mid, v, "right")
    return np.where(lo % 2 == 0, lo, hi)


def bf16_bits(x):
    """bf16 bits of fp64 values that are fp32 numbers, to nearest even."""
    u = np.asarray(x, np.float32).view(np.uint32).astype(np.uint64)
    r = ((u + 0x7fff + ((u >> 16) & 1)) >> 16).astype(np.uint16)
    return np.where(np.isnan(x), np.uint16(0x7fff), r)


def encode(latent, rope):
    """Cache rows [n, row bytes] of latent [n, d_c] and rope [n, d_rope]."""
    n, d_c = latent.shape
    d_rope = rope.shape[1]
    out = np.zeros((n, row_bytes(d_c, d_rope)), np.uint8)
    g = latent.reshape(n, -1, 16)
    ok = np.isfinite(g).all(axis=2)
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        amax = np.where(ok, np.abs(np.where(ok[:, :, None], g, 0)).max(axis=2), 0)
        sb = np.minimum(nearest(amax / 6, SCALES), 247)
        s = SCALES[sb][:, :, None]
        c = nearest(np.where(s > 0, np.abs(np.where(ok[:, :, None], g, 0)) / np.where(s > 0, s, 1), 0), CODES)
        neg = (g < 0) | ((g == 0) & np.signbit(g))
        c = c + 8 * (neg & (s > 0) & ok[:, :, None])
    c = c.reshape(n, -1, 8).astype(np.uint32)
    w = np.zeros(c.shape[:2], np.uint32)
    for e in range(8):
        w |= c[:, :, e] << np.uint32(4 * (e // 2) + 16 * (e % 2))
    out[:, :d_c // 2] = w.astype("<u4").view(np.uint8).reshape(n, -1)
    out[:, d_c // 2:d_c // 2 + 2 * d_rope] = bf16_bits(rope).astype("<u2").view(np.uint8).reshape(n, -1)
    at = d_c // 2 + 2 * d_rope
    out[:, at:at + d_c // 16] = np.where(ok, sb, 255)
    return out


def decode(rows, d_c, d_rope):
    """fp64 values [n, d_c + d_rope] of cache rows."""
    n = rows.shape[0]
    w = np.ascontiguousarray(rows[:, :d_c // 2]).view("<u4").astype(np.uint32)
    c = np.stack([(w >> np.uint32(4 * (e // 2) + 16 * (e % 2))) & 15 for e in range(8)], axis=2).reshape(n, d_c)
    v = np.where(c & 8, -1.0, 1.0) * CODES[c & 7]
    at = d_c // 2 + 2 * d_rope
    sb = rows[:, at:at + d_c // 16]
    s = np.where(sb < 248, SCALES[np.minimum(sb, 247)], np.nan)
    bits = np.ascontiguousarray(rows[:, d_c // 2:at]).view("<u2").astype(np.uint32) << np.uint32(16)
    return np.concatenate([v * np.repeat(s, 16, axis=1), bits.view(np.float32).astype(np.float64)], axis=1)


def rotate(x, angle, interleaved):
    """Rows x [..., d] turned by angle [..., d / 2]."""
    d = x.shape[-1]
    u, v = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :d // 2], x[..., d // 2:])
    z = (u + 1j * v) * np.exp(1j * angle)
    y = np.empty(z.shape[:-1] + (d,))
    if interleaved:
        y[..., 0::2], y[..., 1::2] = z.real, z.imag
    else:
        y[..., :d // 2], y[..., d // 2:] = z.real, z.imag
    return y


class Pool:
    """A block table, its counts and caches, on the host: lists, changed entry by entry."""

    def __init__(self, table, refs, page, caches):
        self.table, self.refs, self.page = [list(r) for r in table], list(refs), page
        self.caches = [c.copy() for c in caches]

    def ok(self, p):
        return 0 <= p < len(self.refs)

    def fork(self, src, dst, lens):
        width, done = len(self.table[0]), set()
        for s, d, L in zip(src, dst, lens):
            first = d not in done
            done.add(d)
            if not (first and s not in dst and 0 <= s < len(self.table) and 0 <= d < len(self.table)
                    and 0 <= L <= width * self.page):
                continue
            n = -(-L // self.page)
            row = [p if self.ok(p) else -1 for p in self.table[s][:n]]
            for p in row:
                if p >= 0:
                    self.refs[p] += 1
            self.table[d] = row + [-1] * (width - n)

    def free(self, rows):
        for r in rows:
            if 0 <= r < len(self.table):
                for p in self.table[r]:
                    if self.ok(p) and self.refs[p] > 0:
                        self.refs[p] -= 1
                self.table[r] = [-1] * len(self.table[r])

    def reserve(self, rows, lens, new):
        """held; pages by the counts at the start."""
        width, page, before = len(self.table[0]), self.page, list(self.refs)
        good, seen = [], set()
        for r, L, N in zip(rows, lens, new):
            g = 0 <= r < len(self.table) and r not in seen and 0 <= L <= N <= width * page
            if 0 <= r < len(self.table):
                seen.add(r)
            if g and L % page and N > L:
                g = self.ok(self.table[r][L // page])
            good.append(g)
        wants = {}
        for i, (r, L, N) in enumerate(zip(rows, lens, new)):
            if good[i] and L % page and N > L and before[self.table[r][L // page]] > 1:
                wants.setdefault(self.table[r][L // page], []).append(i)
        free = [p for p, n in enumerate(before) if n <= 0]
        keeps = {who[0]: p for p, who in wants.items() if len(who) == before[p]}  # all holders are here: the first keeps the page
        needs, served, at = [], [], 0
        for i, (r, L, N) in enumerate(zip(rows, lens, new)):
            need = []
            if good[i] and L % page and N > L and i not in keeps and i in wants.get(self.table[r][L // page], ()):
                need.append(L // page)
            for j in range(-(-L // page), -(-N // page)) if good[i] else ():
                p = self.table[r][j]
                if not (self.ok(p) and before[p] == 1):
                    need.append(j)
            at += len(need)
            needs.append(list(zip(need, free[at - len(need):])))
            served.append(good[i] and (not need or at <= len(free)))
        for i, p in keeps.items():  # it is not its alone while another goes on holding it
            served[i] = served[i] and all(served[k] for k in wants[p][1:])
        changes = []
        for i, (r, L, N) in enumerate(zip(rows, lens, new)):
            for j, to in needs[i] if served[i] else ():
                p = self.table[r][j]
                changes.append((p if self.ok(p) and before[p] > 1 else -1, to))
                self.table[r][j] = to
                if j < -(-L // page):  # the page of held positions
                    for c in self.caches:
                        c[to * page:to * page + L % page] = c[p * page:p * page + L % page]
        for p, to in changes:
            self.refs[to] = 1
            if p >= 0:
                self.refs[p] -= 1
        return [N if s else L for s, L, N in zip(served, lens, new)]

    def compact(self):
        """(moved, live)."""
        live = sum(n > 0 for n in self.refs)
        moved = [p if n > 0 else -1 for p, n in enumerate(self.refs)]
        holes = [p for p in range(live) if self.refs[p] <= 0]
        up = [p for p in range(live, len(self.refs)) if self.refs[p] > 0]
        for s, d in zip(up, holes):
            moved[s] = d
            self.refs[d], self.refs[s] = self.refs[s], 0
            for c in self.caches:
                c[d * self.page:(d + 1) * self.page] = c[s * self.page:(s + 1) * self.page]
        self.table = [[moved[p] if self.ok(p) else -1 for p in r] for r in self.table]
        return moved, live
