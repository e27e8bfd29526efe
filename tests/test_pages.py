"""Pages of a cache: fork, reserve, free, compact, against the entry-by-entry definition."""
import ctypes
import random

import numpy as np
import pytest
import torch

from oracle import kv4_ops as K
from sparse_attention_lightning_gb300 import _abi


def test_oracle_shares_and_copies():
    p = K.Pool([[2, 5], [-1, -1], [-1, -1]], [0, 0, 1, 0, 0, 1], 16, [np.arange(96)])
    p.fork([0, 0], [1, 2], [20, 16])
    assert p.table == [[2, 5], [2, 5], [2, -1]] and p.refs == [0, 0, 3, 0, 0, 2]
    assert p.reserve([1, 2], [20, 16], [21, 17]) == [21, 17]
    assert p.table == [[2, 5], [2, 0], [2, 1]] and p.refs == [1, 1, 3, 0, 0, 1]
    assert list(p.caches[0][:5]) == [80, 81, 82, 83, 4]
    p.free([0])
    assert p.refs == [1, 1, 2, 0, 0, 0] and p.compact() == ([0, 1, 2, -1, -1, -1], 3)
    # all holders of a page in one call: the first keeps it
    p = K.Pool([[1], [1]], [0, 2, 0], 16, [])
    assert p.reserve([1, 0], [3, 3], [4, 4]) == [4, 4] and p.table == [[0], [1]] and p.refs == [1, 1, 0]


def test_argument_checks():
    L = _abi.lib()
    bad, unsup = _abi.DSA_ERR_INVALID_ARG, _abi.DSA_ERR_UNSUPPORTED
    A = [(i + 1) << 28 for i in range(9)]  # addresses far apart
    one = (ctypes.c_void_p * 9)(*A[8:], *[(20 + i) << 28 for i in range(8)])
    row = (ctypes.c_int64 * 9)(*[416] * 9)

    def fork(table=A[0], rows=4, width=8, ld=8, refs=A[1], pages=20, ps=64, n=2, src=A[2], dst=A[3], lens=A[4], ws=A[5],
             wsb=1 << 20):
        return L.dsa_fork_pages(table, rows, width, ld, refs, pages, ps, n, src, dst, lens, ws, wsb, None)

    def free(table=A[0], rows=4, width=8, ld=8, refs=A[1], pages=20, n=2, row=A[2], ws=A[5], wsb=1 << 20):
        return L.dsa_free_pages(table, rows, width, ld, refs, pages, n, row, ws, wsb, None)

    def reserve(table=A[0], rows=4, width=8, ld=8, refs=A[1], pages=20, ps=64, n=2, r=A[2], lens=A[3], new=A[4],
                held=A[6], nc=1, caches=one, rb=row, ws=A[5], wsb=1 << 20):
        return L.dsa_reserve_pages(table, rows, width, ld, refs, pages, ps, n, r, lens, new, held, nc, caches, rb, ws, wsb,
                                   None)

    def compact(table=A[0], rows=4, width=8, ld=8, refs=A[1], pages=20, ps=64, moved=A[2], live=A[3], nc=1, caches=one,
                rb=row, ws=A[5], wsb=1 << 20):
        return L.dsa_compact_pages(table, rows, width, ld, refs, pages, ps, moved, live, nc, caches, rb, ws, wsb, None)

    for f in (fork, free, reserve, compact):
        assert f(table=None) == bad and f(refs=None) == bad and f(table=A[0] + 2) == bad and f(refs=A[1] + 1) == bad
        assert f(rows=0) == bad and f(width=0) == bad and f(ld=7) == bad and f(pages=0) == bad
        assert f(ws=None) == _abi.DSA_ERR_WORKSPACE and f(wsb=100) == _abi.DSA_ERR_WORKSPACE
        assert f(refs=A[0] + 64) == bad  # inside the table
        assert f(rows=1 << 16, width=1 << 15, ld=1 << 15) == unsup
    for f in (fork, reserve, compact):
        assert f(ps=0) == unsup and f(ps=48) == unsup and f(ps=8) == unsup and f(pages=1 << 25) == unsup
    for f in (fork, free, reserve):
        assert f(n=-1) == bad and f(n=0) == _abi.DSA_OK
    assert fork(src=None) == bad and fork(dst=A[3] + 1) == bad and fork(lens=A[0]) == bad and fork(src=A[1] + 4) == bad
    assert free(row=None) == bad and free(row=A[0] + 4) == bad
    assert reserve(held=None) == bad and reserve(held=A[3]) == bad and reserve(new=A[1]) == bad and reserve(r=None) == bad
    assert compact(moved=None) == bad and compact(live=A[2] + 8) == bad
    need = ctypes.c_size_t(0)
    assert L.dsa_pages_workspace_size(4, 2, 20, ctypes.byref(need)) == 0 and reserve(wsb=need.value - 256) == _abi.DSA_ERR_WORKSPACE
    assert L.dsa_pages_workspace_size(0, 2, 20, ctypes.byref(need)) == bad
    for f in (reserve, compact):
        assert f(nc=-1) == unsup and f(nc=9) == unsup and f(caches=None) == bad and f(rb=None) == bad
        assert f(caches=(ctypes.c_void_p * 1)(A[8] + 8)) == bad and f(caches=(ctypes.c_void_p * 1)(None)) == bad
        assert f(rb=(ctypes.c_int64 * 1)(0)) == unsup and f(rb=(ctypes.c_int64 * 1)(1 << 21)) == unsup
        assert f(nc=2, caches=(ctypes.c_void_p * 2)(A[8], A[8])) == bad  # one cache twice
        assert f(caches=(ctypes.c_void_p * 1)(A[1] - 416)) == bad        # the counts inside a cache


class Held:
    """A pool on the GPU beside the oracle's: random rows with shared pages."""

    def __init__(self, rows, width, page, spare, seed, share=0.3, pitch=0):
        r = random.Random(seed)
        self.page, self.rows, self.width = page, rows, width
        self.lens = [r.choice((0, r.randint(0, width * page), r.randint(0, min(width * page, 3 * page)))) for _ in range(rows)]
        pages = sum(-(-n // page) for n in self.lens) + spare
        order = list(range(pages))
        r.shuffle(order)
        table, refs = [], [0] * pages
        for b in range(rows):
            n = -(-self.lens[b] // page)
            row = []
            if b and r.random() < share:  # the head of another row
                row = [p for p in table[r.randrange(b)][:r.randint(0, n)] if p >= 0]
            row += [order.pop() for _ in range(n - len(row))]
            for p in row:
                refs[p] += 1
            table.append(row + [-1] * (width - n))
        g = torch.Generator().manual_seed(seed)
        caches = [torch.randint(0, 256, (pages * page, 416), generator=g, dtype=torch.uint8),
                  torch.randn(pages * page, 9, generator=g), torch.rand(pages * page, generator=g),
                  torch.randint(0, 256, (pages * page, 7), generator=g, dtype=torch.uint8)]
        self.pool = K.Pool(table, refs, page, [c.numpy() for c in caches])
        whole = torch.full((rows, width + pitch), -7, dtype=torch.int32)
        whole[:, :width] = torch.tensor(table, dtype=torch.int32).reshape(rows, width)
        self.whole = whole.cuda()
        self.table, self.refs = self.whole[:, :width], torch.tensor(refs, dtype=torch.int32).cuda()
        self.caches = [c.cuda() for c in caches]
        self.random = r

    def check(self):
        assert self.table.cpu().tolist() == self.pool.table
        assert self.refs.cpu().tolist() == self.pool.refs
        assert (self.whole[:, self.width:] == -7).all()
        for c, want in zip(self.caches, self.pool.caches):
            assert np.array_equal(c.cpu().numpy(), want)

    def i32(self, v):
        return torch.tensor(v, dtype=torch.int32).cuda()


SIZES = [(1, 1, 16, 1, 0), (3, 2, 16, 5, 3), (40, 6, 64, 30, 0), (9, 33, 16, 400, 1), (150, 3, 32, 20, 0), (5, 70, 256, 3, 2)]


@pytest.mark.gpu
@pytest.mark.parametrize("rows,width,page,spare,pitch", SIZES)
@pytest.mark.parametrize("seed", [0, 1])
def test_a_life_of_a_pool(rows, width, page, spare, pitch, seed):
    """Rows freed, forked, reserved and compacted, several times over."""
    import sparse_attention_lightning_gb300 as dsa
    h = Held(rows, width, page, spare, seed + rows, pitch=pitch)
    r, ws = h.random, dsa.Workspace()
    for step in range(4):
        gone = [b for b in range(rows) if r.random() < 0.4] or [0]
        dsa.free_pages(h.table, h.refs, h.i32(gone + gone[:1]), ws=ws)  # the same row twice
        h.pool.free(gone)
        for b in gone:
            h.lens[b] = 0
        h.check()
        stay = [b for b in range(rows) if b not in gone]
        if stay:
            src = [r.choice(stay) for _ in gone]
            lens = [r.choice((h.lens[s], r.randint(0, h.lens[s]))) for s in src]
            dsa.fork_pages(h.table, h.refs, h.i32(src), h.i32(gone), h.i32(lens), page, ws=ws)
            h.pool.fork(src, gone, lens)
            for b, n in zip(gone, lens):
                h.lens[b] = n
            h.check()
        who = r.sample(range(rows), r.randint(1, rows))
        old = [h.lens[b] for b in who]
        new = [min(width * page, n + r.choice((0, 1, r.randint(0, 2 * page)))) for n in old]
        held = dsa.reserve_pages(h.table, h.refs, h.i32(who), h.i32(old), h.i32(new), page, caches=h.caches, ws=ws)
        want = h.pool.reserve(who, old, new)
        assert held.cpu().tolist() == want
        assert ws.status() == (0 if want == new else _abi.DSA_FLAG_NO_PAGES)
        ws.clear_status()
        for b, n in zip(who, want):
            h.lens[b] = n
        h.check()
        moved, live = dsa.compact_pages(h.table, h.refs, page, caches=h.caches, ws=ws)
        assert (moved.cpu().tolist(), int(live)) == h.pool.compact()
        h.check()
        assert ws.status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("free", [0, 1, 2, 3, 9])
def test_too_few_free_pages(free):
    """Entries get all they need in order, or nothing; one that needs nothing is served."""
    import sparse_attention_lightning_gb300 as dsa
    table = [[0, 1, -1], [2, -1, -1], [0, 1, -1], [3, 4, 5]]
    refs = [2, 2, 1, 1, 1, 1] + [0] * free
    caches = [torch.arange(len(refs) * 16, dtype=torch.float32).cuda()]
    pool = K.Pool(table, refs, 16, [c.cpu().numpy() for c in caches])
    t = torch.tensor(table, dtype=torch.int32).cuda()
    n = torch.tensor(refs, dtype=torch.int32).cuda()
    i = lambda v: torch.tensor(v, dtype=torch.int32).cuda()  # noqa: E731
    ws = dsa.Workspace()
    ask = ([0, 1, 2, 3], [20, 16, 20, 40], [21, 48, 40, 40])
    got = dsa.reserve_pages(t, n, i(ask[0]), i(ask[1]), i(ask[2]), 16, caches=caches, ws=ws)
    want = pool.reserve(*ask)
    assert got.cpu().tolist() == want
    assert t.cpu().tolist() == pool.table and n.cpu().tolist() == pool.refs
    assert np.array_equal(caches[0].cpu().numpy(), pool.caches[0])
    assert ws.status() == (_abi.DSA_FLAG_NO_PAGES if want != ask[2] else 0)


@pytest.mark.gpu
def test_a_large_pool():
    """More pages than one round of the counting block, thousands of entries."""
    import sparse_attention_lightning_gb300 as dsa
    h = Held(3000, 24, 16, 20000, 5, share=0.5)
    assert len(h.pool.refs) > 2 * 16384
    r = h.random
    gone = r.sample(range(3000), 1700)
    dsa.free_pages(h.table, h.refs, h.i32(gone))
    h.pool.free(gone)
    stay = sorted(set(range(3000)) - set(gone))
    src = [r.choice(stay) for _ in gone]
    lens = [h.lens[s] for s in src]
    dsa.fork_pages(h.table, h.refs, h.i32(src), h.i32(gone), h.i32(lens), 16)
    h.pool.fork(src, gone, lens)
    for b, n in zip(gone, lens):
        h.lens[b] = n
    who = list(range(3000))
    r.shuffle(who)
    old = [h.lens[b] for b in who]
    new = [min(24 * 16, n + r.randint(0, 40)) for n in old]
    held = dsa.reserve_pages(h.table, h.refs, h.i32(who), h.i32(old), h.i32(new), 16, caches=h.caches)
    assert held.cpu().tolist() == h.pool.reserve(who, old, new)
    h.check()
    moved, live = dsa.compact_pages(h.table, h.refs, 16, caches=h.caches)
    assert (moved.cpu().tolist(), int(live)) == h.pool.compact()
    h.check()


@pytest.mark.gpu
def test_entries_that_make_no_sense_are_left_out():
    import sparse_attention_lightning_gb300 as dsa
    h = Held(6, 4, 16, 30, 3, share=0.0)
    h.lens = [64, 40, 17, 0, 0, 0]
    table = [[0, 1, 2, 3], [4, 5, 99, -1], [6, 7, -1, -1], [-1] * 4, [-1] * 4, [-1] * 4]
    refs = [1] * 8 + [0] * (len(h.pool.refs) - 8)
    h.pool.table, h.pool.refs = [list(r) for r in table], list(refs)
    h.table.copy_(h.i32(table))
    h.refs.copy_(h.i32(refs))
    ws, BAD = dsa.Workspace(), _abi.DSA_FLAG_BAD_INDEX

    def flagged():
        f = ws.status()
        ws.clear_status()
        return f

    for src, dst, lens in (([0, 0], [3, 3], [20, 64]), ([0], [0], [5]), ([0, 3], [3, 4], [16, 16]), ([6], [3], [1]),
                           ([0], [-1], [1]), ([0], [4], [65]), ([0], [4], [-1]), ([1], [5], [40])):
        dsa.fork_pages(h.table, h.refs, h.i32(src), h.i32(dst), h.i32(lens), 16, ws=ws)
        h.pool.fork(src, dst, lens)
        h.check()
        assert flagged() == BAD
    for rows in ([6], [-1], [5, 7, 5]):
        dsa.free_pages(h.table, h.refs, h.i32(rows), ws=ws)
        h.pool.free(rows)
        h.check()
        assert flagged() == BAD
    for who, old, new in (([2, 2], [17, 17], [18, 30]), ([6], [0], [1]), ([2], [18], [17]), ([2], [17], [65]), ([2], [-1], [5]),
                          ([1], [40], [41])):  # the last: its page is none
        held = dsa.reserve_pages(h.table, h.refs, h.i32(who), h.i32(old), h.i32(new), 16, caches=h.caches, ws=ws)
        assert held.cpu().tolist() == h.pool.reserve(who, old, new)
        h.check()
        assert flagged() == BAD
    h.table[5, 0] = h.pool.table[5][0] = len(refs) - 1  # a page that nobody counts as held
    moved, live = dsa.compact_pages(h.table, h.refs, 16, caches=h.caches, ws=ws)
    assert (moved.cpu().tolist(), int(live)) == h.pool.compact()
    assert h.table.cpu().tolist() == h.pool.table and h.pool.table[5] == [-1] * 4
    h.check()
    assert flagged() == BAD


@pytest.mark.gpu
def test_streams_graphs_and_refusals():
    import sparse_attention_lightning_gb300 as dsa
    h = Held(12, 8, 32, 40, 11)
    old, new = h.lens, [min(8 * 32, n + 20) for n in h.lens]
    who = list(range(12))
    args = (h.i32(who), h.i32(old), h.i32(new), 32)
    t0, n0 = h.table.clone(), h.refs.clone()
    pages = len(h.pool.refs)
    need = ctypes.c_size_t(0)
    _abi.check(_abi.lib().dsa_pages_workspace_size(12, 12, pages, ctypes.byref(need)))
    held = torch.zeros(12, dtype=torch.int32).cuda()
    moved, live = torch.zeros(pages, dtype=torch.int32).cuda(), torch.zeros(1, dtype=torch.int32).cuda()
    side = torch.cuda.Stream()

    def step(ws=None):
        dsa.reserve_pages(h.table, h.refs, *args, caches=h.caches, held=held, ws=ws)
        dsa.free_pages(h.table, h.refs, args[0][:3], ws=ws)
        dsa.fork_pages(h.table, h.refs, args[0][3:6], args[0][:3], args[1][3:6], 32, ws=ws)
        dsa.compact_pages(h.table, h.refs, 32, caches=h.caches, moved=moved, live=live, ws=ws)

    graph, ws = torch.cuda.CUDAGraph(), dsa.Workspace(nbytes=need.value)
    torch.cuda.synchronize()
    with pytest.raises(ValueError, match="of its own"):
        with torch.cuda.graph(torch.cuda.CUDAGraph(), stream=side):
            step()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        step(ws)
    caches0 = [c.clone() for c in h.caches]
    for _ in range(2):
        h.table.copy_(t0)
        h.refs.copy_(n0)
        for c, c0 in zip(h.caches, caches0):
            c.copy_(c0)
        graph.replay()
        torch.cuda.synchronize()
        pool = K.Pool(t0.cpu().tolist(), n0.cpu().tolist(), 32, [c.cpu().numpy() for c in caches0])
        assert held.cpu().tolist() == pool.reserve(who, old, new)
        pool.free(who[:3])
        pool.fork(who[3:6], who[:3], old[3:6])
        assert (moved.cpu().tolist(), int(live)) == pool.compact()
        h.pool = pool
        h.check()
    r3 = h.i32([0, 1, 2])
    for bad in (lambda: dsa.free_pages(h.table.long(), h.refs, r3), lambda: dsa.free_pages(h.table.t(), h.refs, r3),
                lambda: dsa.free_pages(h.table, h.refs.long(), r3), lambda: dsa.free_pages(h.table, h.refs.cpu(), r3),
                lambda: dsa.free_pages(h.table, h.refs[::2], r3), lambda: dsa.free_pages(h.table, h.refs, r3.long()),
                lambda: dsa.free_pages(h.table.cpu(), h.refs, r3),
                lambda: dsa.fork_pages(h.table, h.refs, r3, r3[:2], r3, 32),
                lambda: dsa.reserve_pages(h.table, h.refs, r3, r3, r3, 32, caches=[h.caches[0][1:]]),
                lambda: dsa.reserve_pages(h.table, h.refs, r3, r3, r3, 32, caches=[h.caches[0].cpu()]),
                lambda: dsa.reserve_pages(h.table, h.refs, r3, r3, r3, 32, held=r3.long()),
                lambda: dsa.compact_pages(h.table, h.refs, 32, caches=[h.caches[0].t()]),
                lambda: dsa.compact_pages(h.table, h.refs, 32, moved=r3)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(dsa.DsaError):
        dsa.compact_pages(h.table, h.refs, 32, caches=[h.caches[0], h.caches[0]])
    none = r3[:0]
    dsa.free_pages(h.table, h.refs, none)
    dsa.fork_pages(h.table, h.refs, none, none, none, 32)
    assert dsa.reserve_pages(h.table, h.refs, none, none, none, 32).shape == (0,)
    h.check()
