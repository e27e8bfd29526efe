"""Accumulated weight beside entries that are skipped: out of range, ahead of the query, on a page outside the cache."""
import numpy as np
import pytest
import torch

from test_evict import BF, F32, Weights

SHAPES = [(F32, 8, 64, 16), (BF, 16, 64, 16), (BF, 128, 512, 64), (BF, 70, 512, 0)]


def compare(s, idx, lse, flag):
    """The call with `idx` against the definition over s.idx, in which the skipped entries are -1."""
    import sparse_attention_lightning_gb300 as dsa
    n = max(s.case.cfg.k_lens)
    acc = torch.rand(s.case.cfg.num_seqs, n + 5).cuda()
    ref, tol = s.reference(lse, acc)
    got = []
    for entries in (idx, s.idx):
        ws = dsa.Workspace()
        got.append(dsa.accumulate_attn_weights(s.prob, s.q, s.kv, entries.cuda(), lse, acc.clone(), ws=ws))
        assert ws.status() == (flag if entries is idx else 0)
        assert np.all(np.abs(got[-1].double().cpu().numpy() - ref) <= tol)
    assert torch.equal(*got)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,h,d_c,d_rope", SHAPES)
@pytest.mark.parametrize("page", [0, 16])
@pytest.mark.parametrize("q_lens", [[1, 1], [5, 3]])
def test_bad_entries_in_each_place_of_four(q_lens, page, dtype, h, d_c, d_rope):
    """Group g of four entries has bad ones where g has bits; then each value of a bad entry."""
    from sparse_attention_lightning_gb300 import _abi
    for bad in (10 ** 6, -7, -2, 2 ** 31 - 1, -2 ** 31, 300):
        s = Weights(q_lens, [300, 260], h, d_c, d_rope, 130, dtype, page, seed=h)
        mask = torch.tensor([(j // 4 % 16) >> (j % 4) & 1 for j in range(130)], dtype=torch.bool)
        s.idx[:, mask] = -1
        idx = s.idx.clone()
        idx[:, mask] = bad
        compare(s, idx, s.attention(), _abi.DSA_FLAG_BAD_INDEX)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,h,d_c,d_rope", SHAPES)
def test_entries_ahead_of_the_query(dtype, h, d_c, d_rope):
    """Positions that exist, but lie behind the query's own."""
    from sparse_attention_lightning_gb300 import _abi
    s = Weights([6, 4], [200, 90], h, d_c, d_rope, 70, dtype, seed=h)
    idx = s.idx.clone()
    for t, pos in enumerate((194, 195, 196, 197, 198, 199, 86, 87, 88, 89)):
        s.idx[t, t % 4::5] = -1
        idx[t, t % 4::5] = min(pos + 1, 199 if t < 6 else 89) if pos not in (199, 89) else -1
    compare(s, idx, s.attention(), _abi.DSA_FLAG_BAD_INDEX)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,h,d_c,d_rope", SHAPES)
@pytest.mark.parametrize("q_lens", [[1, 1], [5, 3]])
@pytest.mark.parametrize("entry", [-1, 10 ** 6, "num_pages"])
def test_entries_on_pages_outside_the_cache(entry, q_lens, dtype, h, d_c, d_rope):
    from sparse_attention_lightning_gb300 import _abi
    s = Weights(q_lens, [300, 260], h, d_c, d_rope, 130, dtype, 16, seed=h)
    s.prob.block_table[0, 3] = s.prob.num_pages if entry == "num_pages" else entry
    s.prob.block_table[1, ::2] = s.prob.num_pages if entry == "num_pages" else entry
    idx = s.idx.clone()
    first = s.idx[:q_lens[0]]
    first[(first >= 48) & (first < 64)] = -1
    second = s.idx[q_lens[0]:]
    second[(second >= 0) & (second // 16 % 2 == 0)] = -1
    assert not torch.equal(idx, s.idx)
    compare(s, idx, s.attention(), _abi.DSA_FLAG_BAD_INDEX)
