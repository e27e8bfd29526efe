"""Pages reserved for rows that share one, with too few free pages: what a row may write to is its alone."""
import random

import numpy as np
import pytest
import torch

from oracle import kv4_ops as K
from sparse_attention_lightning_gb300 import _abi


def scarce(seed):
    """(pool, entries, lens, new lens): prompts, forks of any length of them, some prompts gone; free pages about as many as wanted."""
    r = random.Random(seed)
    page, width = 16, 4
    prompts, forks = r.randint(1, 4), r.randint(1, 8)
    lens = [r.randint(1, width * page - 3) for _ in range(prompts)] + [0] * forks
    order = list(range(sum(-(-n // page) for n in lens) + r.randint(0, forks + 2)))
    total = len(order)
    r.shuffle(order)
    table = [[order.pop() for _ in range(-(-n // page))] for n in lens]
    refs = [0] * total
    for row in table:
        for p in row:
            refs[p] = 1
        row += [-1] * (width - len(row))
    cache = np.random.default_rng(seed).integers(0, 1 << 30, total * page).astype(np.int32)
    pool = K.Pool(table, refs, page, [cache])
    src = [r.randrange(prompts) for _ in range(forks)]
    cut = [r.choice((lens[s], r.randint(1, lens[s]))) for s in src]
    pool.fork(src, list(range(prompts, prompts + forks)), cut)
    lens[prompts:] = cut
    gone = [b for b in range(prompts) if r.random() < 0.6]
    pool.free(gone)
    for b in gone:
        lens[b] = 0
    who = r.sample(range(len(lens)), r.randint(1, len(lens)))
    old = [lens[b] for b in who]
    new = [min(width * page, n + r.choice((0, 1, 1, 2, 20))) for n in old]
    return pool, lens, who, old, new


def check_alone(table, refs, page, who, old, held):
    """No page of positions old .. held - 1 of an entry's row has another holder, and the counts are the table's."""
    holders = {}
    for row in table:
        for p in row:
            if p >= 0:
                holders[p] = holders.get(p, 0) + 1
    assert [holders.get(p, 0) for p in range(len(refs))] == refs
    for b, L, N in zip(who, old, held):
        for j in range(L // page, -(-N // page)) if N > L else ():
            assert holders[table[b][j]] == 1, (b, j)


def test_a_page_is_kept_only_by_its_last_holder():
    """One page, no free one: neither of two rows may write to it, whichever is longer.  With a free one both may."""
    for lens in ([10, 14], [14, 10], [5, 12], [7, 7]):
        new = [n + 1 for n in lens]
        p = K.Pool([[0], [0]], [2], 16, [])
        assert p.reserve([1, 0], lens, new) == lens and p.table == [[0], [0]] and p.refs == [2]
        p = K.Pool([[0], [0]], [2, 0], 16, [])
        assert p.reserve([1, 0], lens, new) == new and p.table == [[1], [0]] and p.refs == [1, 1]


def test_definition_leaves_no_shared_page_to_write_to():
    short = 0
    for seed in range(2000):
        pool, _, who, old, new = scarce(seed)
        held = pool.reserve(who, old, new)
        check_alone(pool.table, pool.refs, pool.page, who, old, held)
        short += held != new
    assert 200 < short < 1900


@pytest.mark.gpu
@pytest.mark.parametrize("block", range(8))
def test_rows_write_without_touching_others(block):
    """Against the definition; then every row writes the positions that it got, and every other row's positions keep their bytes."""
    import sparse_attention_lightning_gb300 as dsa
    i32 = lambda v: torch.tensor(v, dtype=torch.int32).cuda()  # noqa: E731
    ws = dsa.Workspace()
    for seed in range(40 * block, 40 * block + 40):
        pool, lens, who, old, new = scarce(seed)
        page = pool.page
        table, refs, cache = i32(pool.table), i32(pool.refs), torch.from_numpy(pool.caches[0].copy()).cuda()
        rows = lambda t, b, n: [t[b][s // page] * page + s % page for s in range(n)]  # noqa: E731
        before = [pool.caches[0][rows(pool.table, b, lens[b])] for b in range(len(lens))]
        held = dsa.reserve_pages(table, refs, i32(who), i32(old), i32(new), page, caches=[cache], ws=ws).cpu().tolist()
        assert held == pool.reserve(who, old, new), seed
        assert ws.status() == (0 if held == new else _abi.DSA_FLAG_NO_PAGES)
        ws.clear_status()
        t, got = table.cpu().tolist(), cache.cpu().numpy()
        assert t == pool.table and refs.cpu().tolist() == pool.refs and np.array_equal(got, pool.caches[0])
        check_alone(t, refs.cpu().tolist(), page, who, old, held)
        for b, L, N in zip(who, old, held):
            got[rows(t, b, N)[L:]] = -1 - b
        for b in range(len(lens)):
            assert np.array_equal(got[rows(t, b, lens[b])], before[b]), (seed, b)


@pytest.mark.gpu
@pytest.mark.parametrize("free", [0, 1, 700, 1399, 1400])
def test_thousands_of_pairs_with_too_few_pages(free):
    """1,400 pairs of rows that share a page, all in the call: as many pairs as there are free pages are served."""
    import sparse_attention_lightning_gb300 as dsa
    i32 = lambda v: torch.tensor(v, dtype=torch.int32).cuda()  # noqa: E731
    r = random.Random(free)
    n = 1400
    table, refs = [[b % n] for b in range(2 * n)], [2] * n + [0] * free
    lens = [r.randint(1, 15) for _ in range(2 * n)]
    who = r.sample(range(2 * n), 2 * n)
    old = [lens[b] for b in who]
    new = [k + 1 for k in old]
    pool = K.Pool(table, refs, 16, [np.arange(16 * len(refs), dtype=np.int32)])
    t, c, cache = i32(table), i32(refs), torch.from_numpy(pool.caches[0].copy()).cuda()
    held = dsa.reserve_pages(t, c, i32(who), i32(old), i32(new), 16, caches=[cache]).cpu().tolist()
    assert held == pool.reserve(who, old, new) and sum(h > o for h, o in zip(held, old)) == 2 * free
    assert t.cpu().tolist() == pool.table and c.cpu().tolist() == pool.refs
    assert np.array_equal(cache.cpu().numpy(), pool.caches[0])
    check_alone(pool.table, pool.refs, 16, who, old, held)
