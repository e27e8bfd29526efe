"""Accumulated weight where a CTA of the tensor-core kernel works on several chunks of a query, on several queries, and
starts in the middle of one."""
import pytest
import torch

from test_evict import BF, Weights


def shares(total_q, top_k):
    """(pieces a query is split into, consecutive ones a CTA takes): the launcher's choice on this GPU."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    chunks = -(-top_k // 64)
    best = None
    for s in range(1, chunks + 1):
        n = -(-total_q * s // sms)
        blocks = 1 if s % n == 0 else n // s if n % s == 0 else (n - 2) // s + 2
        cost = (n * chunks + s - 1) // s + 2 * blocks
        if best is None or cost < best[0]:
            best = cost, s, n
    return best[1:]


def run_twice(s):
    import sparse_attention_lightning_gb300 as dsa
    before, lse, got = s.check()
    for _ in range(2):
        ws = dsa.Workspace()
        again = dsa.accumulate_attn_weights(s.prob, s.q, s.kv, s.idx.cuda(), lse, before.clone(), ws=ws)
        assert torch.equal(got, again) and ws.status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("h,d_c,d_rope,page", [(128, 512, 64, 0), (16, 512, 64, 64), (128, 64, 16, 16), (40, 64, 0, 0)])
@pytest.mark.parametrize("queries", [36, 150])
def test_many_chunks_a_cta(queries, h, d_c, d_rope, page):
    """One query a sequence; 8 chunks a CTA for 36 queries of 2048 positions, 32 for 150."""
    split, per = shares(queries, 2048)
    assert per * (32 // split) >= 8
    k_lens = [2048 + 13 * (i % 7) - (1700 if i % 5 == 2 else 0) for i in range(queries)]
    run_twice(Weights([1] * queries, k_lens, h, d_c, d_rope, 2048, BF, page, seed=queries + h))


@pytest.mark.gpu
@pytest.mark.parametrize("h,d_c,d_rope", [(128, 512, 64), (16, 512, 64), (128, 64, 16), (16, 64, 0)])
@pytest.mark.parametrize("q_lens,k", [([100, 100], 500), ([190, 3, 0, 150, 1], 65)])
def test_several_queries_a_cta(q_lens, k, h, d_c, d_rope):
    """Query blocks loaded again, shares that begin in mid-query."""
    split, per = shares(sum(q_lens), k)
    assert per > split or per % split  # CTAs with more than one query
    run_twice(Weights(q_lens, [700 + T for T in q_lens], h, d_c, d_rope, k, BF, seed=k + h))


@pytest.mark.gpu
@pytest.mark.parametrize("h,d_c,d_rope", [(16, 512, 64), (128, 512, 64), (64, 64, 16), (100, 64, 16)])
@pytest.mark.parametrize("T,n,k", [(1, 600, 100), (1, 608, 40), (20, 15, 130)])
def test_refused_queries_between_good_ones(T, n, k, h, d_c, d_rope):
    """Sequences with more queries than positions: their rows stay as they were, the others' get the same bytes.  (Paged:
    a longer neighbour keeps its rows.)"""
    import sparse_attention_lightning_gb300 as dsa
    from sparse_attention_lightning_gb300 import _abi
    split, per = shares(T * n, k)
    assert per > split
    s = Weights([T] * n, [90] * (n - 1) + [900], h, d_c, d_rope, k, BF, 16, seed=T + h)
    lse, idx, acc0 = s.attention(), s.idx.cuda(), torch.rand(n, 900).cuda()
    ref = dsa.accumulate_attn_weights(s.prob, s.q, s.kv, idx, lse, acc0.clone())
    cu = s.prob.cu_k.cpu()
    refused = [b for b in range(n - 4) if b % 9 in (2, 3, 4, 5) or (T > 1 and b % 3 == 1)]
    for b in range(n - 1):  # refused sequences hold T - 1 positions, the next good one what is left over
        if b in refused:
            cu[b + 1] = cu[b] + T - 1
    s.prob.cu_k.copy_(cu)
    for _ in range(4):
        ws = dsa.Workspace()
        got = dsa.accumulate_attn_weights(s.prob, s.q, s.kv, idx, lse, acc0.clone(), ws=ws)
        assert ws.status() == _abi.DSA_FLAG_BAD_SEQS
        for b in range(n):
            want = acc0[b] if b in refused else ref[b]
            assert torch.equal(got[b], want), b
