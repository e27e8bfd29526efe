"""A workspace that grows: what earlier calls and captured graphs use stays theirs, and memory stays bounded."""
import pytest
import torch

from test_prefix_attn import BF, FULL, Setup


def test_earlier_buffers_stay_and_stay_few():
    import sparse_attention_lightning_gb300 as dsa
    ws = dsa.Workspace("cpu")
    ws.buf[3] = 5  # a status flag
    bufs = [ws.buf]
    for n in range(dsa._abi.STATUS_BYTES, 40 * dsa._abi.STATUS_BYTES, 1000):  # a little more each call
        assert ws.ensure(n) is ws and ws.nbytes >= n
        if ws.buf is not bufs[-1]:
            assert int(ws.buf[3]) == 5 and int(ws.buf.sum()) == 5
            bufs.append(ws.buf)
    assert len(bufs) <= 7
    held = ws._earlier
    assert [b.data_ptr() for b in held] == [b.data_ptr() for b in bufs[:-1]]
    assert sum(b.numel() for b in held) < ws.nbytes


@pytest.mark.gpu
def test_graph_keeps_its_buffer_when_another_operator_grows_the_workspace():
    """Captured with one operator; the workspace then grows in fused_forward."""
    import sparse_attention_lightning_gb300 as dsa
    from sparse_attention_lightning_gb300 import _abi
    from sparse_attention_lightning_gb300 import workloads as W
    s = Setup([1, 1], [30, 60], 16, P=2000, dtype=BF, seed=14, **FULL)
    q = s.q.cuda()
    ws = dsa.Workspace(nbytes=s.prob.workspace_size(_abi.OP_PREFIX_MLA_ATTN))
    ref, ref_lse = s.run()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out, lse = dsa.prefix_mla_attn(s.prob, q, s.kv, ws=ws, **s.prefix)
    held, room = ws.buf.data_ptr(), ws.nbytes
    cfg = W.custom([400], [9000], idx_dtype="bf16", kv_dtype="bf16", top_k=64)
    d = {k: v.cuda() for k, v in W.make_case(cfg, 1).tensors().items()}
    P = dsa.Problem.from_config(cfg, d["cu_q"], d["cu_k"])
    assert P.workspace_size(_abi.OP_FUSED_FORWARD) > room
    first = dsa.fused_forward(P, d["q_idx"], d["k_idx"], d["w"], d["q"], d["kv"], ws=ws)
    assert ws.buf.data_ptr() != held
    junk = [torch.full((room // 4,), 255, dtype=torch.uint8, device="cuda") for _ in range(64)]
    junk += [torch.full((room,), 255, dtype=torch.uint8, device="cuda") for _ in range(8)]
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ref) and torch.equal(lse, ref_lse)
    assert all((j == 255).all() for j in junk)
    again = dsa.fused_forward(P, d["q_idx"], d["k_idx"], d["w"], d["q"], d["kv"], ws=ws)
    assert all(torch.equal(x, y) for x, y in zip(first[:3], again[:3])) and ws.status() == 0


@pytest.mark.gpu
def test_workspace_grows_behind_a_call_on_another_stream():
    """A call in flight on a side stream keeps its scratch while the next, ordered behind it, grows the workspace."""
    import sparse_attention_lightning_gb300 as dsa
    s = Setup([1, 1], [30, 60], 16, P=9000, dtype=BF, seed=3, **FULL)
    big = Setup([1] * 9, [60] * 9, 128, P=2000, dtype=BF, seed=15, **FULL)
    q, q2 = s.q.cuda(), big.q.cuda()
    want, want2 = s.run(), big.run()
    for _ in range(5):
        ws = dsa.Workspace()
        a, b = torch.cuda.Stream(), torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.stream(a):
            torch.cuda._sleep(2_000_000)
            got = dsa.prefix_mla_attn(s.prob, q, s.kv, ws=ws, **s.prefix)
        b.wait_stream(a)
        with torch.cuda.stream(b):
            got2 = dsa.prefix_mla_attn(big.prob, q2, big.kv, ws=ws, **big.prefix)
        junk = torch.full((1 << 24,), 255, dtype=torch.uint8, device="cuda")  # on the default stream, at once
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip((*got, *got2), (*want, *want2)))
        assert (junk == 255).all() and ws.status() == 0
