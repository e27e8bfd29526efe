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
