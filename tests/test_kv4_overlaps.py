"""dsa_sparse_mla_attn4 refuses outputs that lie over its inputs or each other: a query's output would be written while another
query's inputs there are still read."""
import ctypes

from sparse_attention_lightning_gb300 import _abi


def test_outputs_over_inputs_are_refused():
    L, A, bad, wse = _abi.lib(), 1 << 24, _abi.DSA_ERR_INVALID_ARG, _abi.DSA_ERR_WORKSPACE
    p = _abi.DsaProblem(num_seqs=1, total_q=4, total_k=64, max_q_len=4, max_k_len=64, h_idx=4, d_idx=32, h=8, d_c=64, d_rope=16, top_k=8,
                        idx_dtype=0, kv_dtype=_abi.DSA_BF16, out_dtype=_abi.DSA_F32, sm_scale=0.0, cu_q=4096, cu_k=8192)
    q_bytes, kv4_bytes, idx_bytes, out_bytes, lse_bytes = 4 * 8 * 80 * 2, 64 * 80, 4 * 8 * 4, 4 * 8 * 64 * 4, 4 * 8 * 4

    def attn(out=4 * A, lse=5 * A, q=A, kv4=2 * A, idx=3 * A):  # (without a workspace: nothing is launched)
        return L.dsa_sparse_mla_attn4(ctypes.byref(p), q, kv4, idx, out, lse, None, 0, None)

    assert attn() == wse and attn(lse=None) == wse and attn(q=3 * A, idx=3 * A) == wse
    for at, size in ((A, q_bytes), (2 * A, kv4_bytes), (3 * A, idx_bytes)):
        for f, own in ((lambda v: attn(out=v), out_bytes), (lambda v: attn(lse=v), lse_bytes)):
            assert f(at) == bad and f(at + size - 16) == bad and f(at - own + 16) == bad
            assert f(at + size) == wse and f(at - own) == wse
    assert attn(lse=4 * A + 64) == bad and attn(lse=4 * A + out_bytes) == wse
