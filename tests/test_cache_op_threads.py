"""The operators around the caches called by several host threads."""
import threading

import pytest
import torch

from test_evict import BF, F32, Weights
from test_prefix_attn import Setup


def in_threads(*bodies):
    """Run the bodies side by side from one starting line; the first exception is raised here."""
    start, failed = threading.Barrier(len(bodies)), []

    def run(body):
        try:
            start.wait()
            body()
        except BaseException as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=run, args=(b,)) for b in bodies]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    if failed:
        raise failed[0]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
def test_threads_with_different_widths(dtype):
    """Narrow and wide rows launch the same kernels with different amounts of shared memory."""
    import sparse_attention_lightning_gb300 as dsa
    bodies, bad = [], []
    for d_c, d_rope in ((64, 0), (1024, 256), (512, 64)):
        w = Weights([1, 1], [40, 30], 4, d_c, d_rope, 24, dtype, seed=d_c)
        lse, idx = w.attention(), w.idx.cuda()
        s = Setup([1, 2], [20, 9], 4, d_c, d_rope, 70, dtype, seed=d_c)
        q, stream = s.q.cuda(), torch.cuda.Stream()
        want = (dsa.accumulate_attn_weights(w.prob, w.q, w.kv, idx, lse, torch.zeros(2, 40).cuda()),
                *dsa.prefix_mla_attn(s.prob, q, s.kv, **s.prefix))
        torch.cuda.synchronize()

        def body(w=w, lse=lse, idx=idx, s=s, q=q, stream=stream, want=want):
            with torch.cuda.stream(stream):
                for _ in range(300):
                    got = (dsa.accumulate_attn_weights(w.prob, w.q, w.kv, idx, lse,
                                                       torch.zeros(2, 40, device="cuda")),
                           *dsa.prefix_mla_attn(s.prob, q, s.kv, **s.prefix))
                stream.synchronize()
                bad.extend(not torch.equal(g, x) for g, x in zip(got, want))

        bodies.append(body)
    in_threads(*bodies)
    assert len(bad) == 9 and not any(bad)


def test_default_workspaces_belong_to_a_thread_and_a_stream(monkeypatch):
    """Threads on one stream, with no GPU: a call's scratch is handed out again to its own thread alone."""
    import sparse_attention_lightning_gb300 as dsa

    class Fake:
        def __init__(self, device, nbytes):
            self.nbytes = nbytes

    monkeypatch.setattr(dsa, "Workspace", Fake)
    monkeypatch.setattr(dsa, "_capturing", lambda: False)
    got = [[], []]

    def body(mine):
        for _ in range(3):
            mine += [dsa._op_workspace(None, 0, 7, 100), dsa._op_workspace(None, 0, 9, 100)]
        mine.append(dsa._op_workspace(None, 0, 7, 101))

    in_threads(*[lambda m=m: body(m) for m in got])
    for mine in got:
        assert len({id(w) for w in mine[::2][:3]}) == 1 and len({id(w) for w in mine[1::2]}) == 1
        assert mine[0] is not mine[1] and mine[6] is not mine[0] and mine[6].nbytes == 200
    assert not {id(w) for w in got[0]} & {id(w) for w in got[1]}


@pytest.mark.gpu
def test_threads_on_one_stream():
    """An operator is two or three launches that share its scratch; two threads' launches may alternate on the stream."""
    import sparse_attention_lightning_gb300 as dsa
    bodies, bad = [], []
    for seed in (1, 2, 3):
        w = Weights([9, 30], [600, 800], 16, 64, 16, 200, BF, seed=seed)
        lse, idx = w.attention(), w.idx.cuda()
        s = Setup([1, 1], [20, 90], 16, 512, 64, 2000, BF, seed=seed)
        q = s.q.cuda()
        w.check(lse=lse)
        s.check(*s.run())
        want = (dsa.accumulate_attn_weights(w.prob, w.q, w.kv, idx, lse, torch.zeros(2, 800).cuda()),
                *dsa.prefix_mla_attn(s.prob, q, s.kv, **s.prefix))

        def body(w=w, lse=lse, idx=idx, s=s, q=q, want=want):
            for _ in range(100):
                got = (dsa.accumulate_attn_weights(w.prob, w.q, w.kv, idx, lse,
                                                   torch.zeros(2, 800, device="cuda")),
                       *dsa.prefix_mla_attn(s.prob, q, s.kv, **s.prefix))
                bad.extend(not torch.equal(g, x) for g, x in zip(got, want))

        bodies.append(body)
    torch.cuda.synchronize()
    in_threads(*bodies)
    assert len(bad) == 900 and not any(bad)


@pytest.mark.gpu
@pytest.mark.parametrize("q_lens", [[1, 1], [70, 5]])
def test_weights_on_two_streams(q_lens):
    """Calls on two streams at once, with default scratch and as graphs with a workspace each, behind a wait that lets
    both start together."""
    import sparse_attention_lightning_gb300 as dsa
    from sparse_attention_lightning_gb300 import _abi
    sets = []
    for seed in (1, 2):
        w = Weights(q_lens, [3000, 900], 128, 512, 64, 700, BF, seed=seed)
        lse, idx = w.attention(), w.idx.cuda()
        want = dsa.accumulate_attn_weights(w.prob, w.q, w.kv, idx, lse, torch.zeros(2, 3000).cuda())
        sets.append((w, lse, idx, want, torch.cuda.Stream(), torch.zeros(2, 3000).cuda()))
    for _ in range(10):
        torch.cuda.synchronize()
        for w, lse, idx, want, st, acc in sets:
            with torch.cuda.stream(st):
                torch.cuda._sleep(200_000)
                acc.zero_()
                dsa.accumulate_attn_weights(w.prob, w.q, w.kv, idx, lse, acc)
        torch.cuda.synchronize()
        assert all(torch.equal(acc, want) for _, _, _, want, _, acc in sets)
    graphs = []
    for w, lse, idx, want, st, acc in sets:
        ws = dsa.Workspace(nbytes=w.prob.workspace_size(_abi.OP_ATTN_WEIGHTS))
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            acc.zero_()
            dsa.accumulate_attn_weights(w.prob, w.q, w.kv, idx, lse, acc, ws=ws)
        graphs.append((graph, ws))
    for _ in range(10):
        torch.cuda.synchronize()
        for (graph, _ws), s in zip(graphs, sets):
            with torch.cuda.stream(s[4]):
                torch.cuda._sleep(200_000)
                graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(acc, want) for _, _, _, want, _, acc in sets)
