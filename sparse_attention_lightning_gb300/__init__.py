"""GB300 (sm_103a) DSA hot path: Lightning Indexer → Top-K → sparse MLA attention.

A thin binding over libdsa.so (include/dsa.h).  Functions take CUDA tensors,
check their dtypes and shapes, and pass raw pointers plus the current CUDA
stream to the library; every step of the computation runs in the library's
kernels.  There is no CPU or framework fallback: if the library is missing,
calls raise.

Names follow the C ABI: indexer_scores, topk, fused_indexer, sparse_mla_attn,
fused_forward, indexer_prolog, add_rmsnorm, prefix_mla_attn, accumulate_attn_weights, evict,
rotate_axes, write_kv4, read_kv4, sparse_mla_attn4, fork_pages, free_pages, reserve_pages, compact_pages.
"""
from __future__ import annotations

import array
import ctypes
import math
import threading
from typing import NamedTuple, Optional, Sequence, Tuple

import torch

from . import _abi
from ._abi import STATUS_BYTES, DsaError, lib  # noqa: F401

__all__ = ["Problem", "Workspace", "indexer_scores", "topk", "fused_indexer", "sparse_mla_attn",
           "fused_forward", "indexer_prolog", "add_rmsnorm", "prefix_mla_attn",
           "accumulate_attn_weights", "evict", "Eviction", "Rotary", "rotate_axes", "kv4_row_bytes",
           "write_kv4", "read_kv4", "sparse_mla_attn4", "fork_pages", "free_pages", "reserve_pages",
           "compact_pages", "DsaError", "lib", "trace"]

_DT = {torch.float32: _abi.DSA_F32, torch.bfloat16: _abi.DSA_BF16,
       torch.uint8: _abi.DSA_FP8_E4M3, torch.float8_e4m3fn: _abi.DSA_FP8_E4M3}
_NAME_DT = {"f32": _abi.DSA_F32, "bf16": _abi.DSA_BF16, "e4m3": _abi.DSA_FP8_E4M3,
            "mxfp8": _abi.DSA_MXFP8_E4M3}
_TORCH_OUT = {_abi.DSA_F32: torch.float32, _abi.DSA_BF16: torch.bfloat16}


def _dt(x) -> int:
    if isinstance(x, str):
        return _NAME_DT[x]
    if isinstance(x, int):
        return x
    return _DT[x]


class Problem:
    """Sizes, dtypes and device sequence offsets of one DSA problem (dsa_problem)."""

    def __init__(self, cu_q: torch.Tensor, cu_k: torch.Tensor, *, q_lens: Sequence[int],
                 k_lens: Sequence[int], h_idx: int, d_idx: int, h: int, d_c: int, d_rope: int,
                 top_k: int, idx_dtype, kv_dtype, out_dtype=None, sm_scale: float = 0.0,
                 block_table: Optional[torch.Tensor] = None, page_size: int = 0,
                 num_pages: int = 0):
        """block_table [B, max_pages] int32 (CUDA) with page_size > 0 and num_pages: the key
        caches (k_idx, kv, k_scale) are paged, num_pages * page_size rows; key position s of
        sequence b is row block_table[b, s // page_size] * page_size + s % page_size.
        Calls read block_table as it is when they run, so pages reserved later are seen; a table
        whose rows are apart is copied (contiguously), and the copy stays as it was."""
        if not (cu_q.is_cuda and cu_k.is_cuda) or cu_q.dtype != torch.int32 \
                or cu_k.dtype != torch.int32:
            raise ValueError("cu_q/cu_k must be int32 CUDA tensors")
        self.cu_q, self.cu_k = cu_q.contiguous(), cu_k.contiguous()
        self.page_size, self.num_pages = int(page_size), int(num_pages)
        self.block_table = None
        if self.page_size:
            if block_table is None or not block_table.is_cuda or block_table.dtype != torch.int32 \
                    or block_table.dim() != 2 or block_table.shape[0] != len(q_lens):
                raise ValueError("paged caches need an int32 CUDA block_table [B, max_pages]")
            self.block_table = block_table.contiguous()
        self.q_lens, self.k_lens = list(q_lens), list(k_lens)
        self.h_idx, self.d_idx, self.h, self.d_c, self.d_rope = h_idx, d_idx, h, d_c, d_rope
        self.top_k = top_k
        self.idx_dtype, self.kv_dtype = _dt(idx_dtype), _dt(kv_dtype)
        self.out_dtype = _dt(out_dtype) if out_dtype is not None else self.kv_dtype
        self.sm_scale = float(sm_scale)
        self.c = _abi.DsaProblem(
            len(self.q_lens), sum(self.q_lens), sum(self.k_lens), max(self.q_lens, default=0),
            max(self.k_lens), h_idx, d_idx, h, d_c, d_rope, top_k, self.idx_dtype, self.kv_dtype,
            self.out_dtype, self.sm_scale, self.cu_q.data_ptr(), self.cu_k.data_ptr(),
            self.page_size, self.block_table.shape[1] if self.page_size else 0, self.num_pages,
            self.block_table.data_ptr() if self.page_size else None)
        self._ref = ctypes.byref(self.c)
        # what the operators around the caches check a call's tensors against
        self._ws_sizes = {}
        self._row_specs = None
        tq = self.c.total_q
        self._shapes = ((tq, h, self.d), (self.cache_rows, self.d), (tq, h, d_c), (tq, h), (tq, top_k))
        self._device = self.cu_q.get_device()
        if any(t.get_device() != self._device for t in (self.cu_k, self.block_table) if t is not None):
            raise ValueError("cu_q, cu_k and block_table must be on one device")

    @classmethod
    def from_config(cls, cfg, cu_q: torch.Tensor, cu_k: torch.Tensor, sm_scale: float = 0.0,
                    block_table: Optional[torch.Tensor] = None, page_size: int = 0,
                    num_pages: int = 0):
        return cls(cu_q, cu_k, q_lens=cfg.q_lens, k_lens=cfg.k_lens, h_idx=cfg.h_idx,
                   d_idx=cfg.d_idx, h=cfg.h, d_c=cfg.d_c, d_rope=cfg.d_rope, top_k=cfg.top_k,
                   idx_dtype=cfg.idx_dtype, kv_dtype=cfg.kv_dtype, out_dtype=cfg.out_dtype,
                   sm_scale=sm_scale, block_table=block_table, page_size=page_size,
                   num_pages=num_pages)

    @property
    def cache_rows(self) -> int:
        """Rows of the key caches (k_idx, kv, k_scale)."""
        return self.num_pages * self.page_size if self.page_size else self.total_k

    @property
    def total_q(self) -> int:
        return self.c.total_q

    @property
    def total_k(self) -> int:
        return self.c.total_k

    @property
    def max_k_len(self) -> int:
        return self.c.max_k_len

    @property
    def d(self) -> int:
        return self.d_c + self.d_rope

    @property
    def scale(self) -> float:
        return self.sm_scale if self.sm_scale > 0 else 1.0 / math.sqrt(self.d)

    def workspace_size(self, op: int) -> int:
        n = ctypes.c_size_t(0)
        _abi.check(lib().dsa_workspace_size(ctypes.byref(self.c), op, ctypes.byref(n)))
        return n.value


class Workspace:
    """Caller-owned device scratch; its first 16384 bytes are the status block (the status
    word and the kernels' synchronisation counters, zero between calls).

    A call that needs more than the workspace holds gives it a new buffer, of at least twice the size, with the
    status block carried over.  Earlier buffers live as long as the workspace (together they are smaller than the
    current one): captured graphs may refer to them, and calls on other streams may still use them.  A graph's kernels go on
    reporting into the buffer that the graph was captured with."""

    def __init__(self, device=None, nbytes: int = STATUS_BYTES):
        self.device = torch.device(device or "cuda")
        self.buf = torch.zeros(max(STATUS_BYTES, nbytes), dtype=torch.uint8, device=self.device)
        self._earlier = []

    def ensure(self, nbytes: int) -> "Workspace":
        held = self.buf.numel()
        if held < nbytes:
            grown = torch.zeros(max(nbytes, 2 * held), dtype=torch.uint8, device=self.device)
            grown[:STATUS_BYTES].copy_(self.buf[:STATUS_BYTES])
            self._earlier.append(self.buf)
            self.buf = grown
        return self

    @property
    def ptr(self) -> int:
        return self.buf.data_ptr()

    @property
    def nbytes(self) -> int:
        return self.buf.numel()

    def clear_status(self) -> None:
        _abi.check(lib().dsa_clear_status(self.ptr, _stream(self.device)))

    def selftest_wait_timeout(self, limit_ns: int = 1_000_000) -> None:
        """Run the bounded-wait self-test: a wait on an mbarrier nothing arrives at gives up
        after limit_ns and sets DSA_FLAG_TIMEOUT in this workspace's status word."""
        _abi.check(lib().dsa_selftest_wait_timeout(self.ptr, int(limit_ns), _stream(self.device)))

    def status(self) -> int:
        """Synchronise the current stream and return the device status flags."""
        f = ctypes.c_uint32(0)
        rc = lib().dsa_read_status(self.ptr, _stream(self.device), ctypes.byref(f))
        if rc not in (_abi.DSA_OK, _abi.DSA_ERR_TIMEOUT):
            _abi.check(rc)
        return f.value


_default_ws = {}


def _workspace(ws: Optional[Workspace], device, nbytes: int) -> Workspace:
    if ws is None:
        key = torch.device(device).index
        ws = _default_ws.get(key)
        if ws is None:
            ws = _default_ws[key] = Workspace(device, nbytes)
    return ws.ensure(nbytes)


def _stream(device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _need(t: Optional[torch.Tensor], name: str, dtype_code: Optional[int], shape: Tuple[int, ...],
          optional: bool = False) -> None:
    if t is None:
        if optional:
            return
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype_code is not None and _DT.get(t.dtype) != dtype_code:
        raise ValueError(f"{name} has dtype {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _check_indexer(P: Problem, q_idx, k_idx, w, q_scale, k_scale):
    mx = P.idx_dtype == _abi.DSA_MXFP8_E4M3
    codes = _abi.DSA_FP8_E4M3 if mx else P.idx_dtype  # MXFP8 codes are E4M3 bytes
    _need(q_idx, "q_idx", codes, (P.total_q, P.h_idx, P.d_idx))
    _need(k_idx, "k_idx", codes, (P.cache_rows, P.d_idx))
    _need(w, "w", _abi.DSA_F32, (P.total_q, P.h_idx))
    if mx:  # E8M0 bytes, one per 32 elements
        _need(q_scale, "q_scale", _abi.DSA_FP8_E4M3, (P.total_q, P.h_idx, P.d_idx // 32))
        _need(k_scale, "k_scale", _abi.DSA_FP8_E4M3, (P.cache_rows, P.d_idx // 32))
        return
    fp8 = P.idx_dtype == _abi.DSA_FP8_E4M3
    _need(q_scale, "q_scale", _abi.DSA_F32, (P.total_q, P.h_idx), optional=not fp8)
    _need(k_scale, "k_scale", _abi.DSA_F32, (P.cache_rows,), optional=not fp8)


def _idx_out(P: Problem, idx, vals, device, want_vals: bool):
    if idx is None:
        idx = torch.empty(P.total_q, P.top_k, dtype=torch.int32, device=device)
    _need(idx, "idx", None, (P.total_q, P.top_k))
    if vals is None and want_vals:
        vals = torch.empty(P.total_q, P.top_k, dtype=torch.float32, device=device)
    _need(vals, "vals", _abi.DSA_F32, (P.total_q, P.top_k), optional=True)
    return idx, vals


def indexer_scores(P: Problem, q_idx, k_idx, w, q_scale=None, k_scale=None, scores=None,
                   ws: Optional[Workspace] = None) -> torch.Tensor:
    """scores[ΣT, max_k_len] (fp32, -inf past each query's position)."""
    _check_indexer(P, q_idx, k_idx, w, q_scale, k_scale)
    dev = k_idx.device
    if scores is None:
        scores = torch.empty(P.total_q, P.max_k_len, dtype=torch.float32, device=dev)
    _need(scores, "scores", _abi.DSA_F32, (P.total_q, scores.shape[1]))
    ws = _workspace(ws, dev, P.workspace_size(_abi.OP_INDEXER_SCORES))
    _abi.check(lib().dsa_indexer_scores(
        ctypes.byref(P.c), q_idx.data_ptr(), k_idx.data_ptr(), w.data_ptr(), _ptr(q_scale),
        _ptr(k_scale), scores.data_ptr(), scores.shape[1], ws.ptr, ws.nbytes, _stream(dev)))
    return scores


def topk(P: Problem, scores: torch.Tensor, idx=None, vals=None, want_vals: bool = False,
         ws: Optional[Workspace] = None):
    """(idx[ΣT, top_k] int32 ascending positions, -1 padded; vals or None)."""
    _need(scores, "scores", _abi.DSA_F32, (P.total_q, scores.shape[1]))
    dev = scores.device
    idx, vals = _idx_out(P, idx, vals, dev, want_vals)
    ws = _workspace(ws, dev, P.workspace_size(_abi.OP_TOPK))
    _abi.check(lib().dsa_topk(ctypes.byref(P.c), scores.data_ptr(), scores.shape[1],
                              idx.data_ptr(), _ptr(vals), ws.ptr, ws.nbytes, _stream(dev)))
    return idx, vals


def fused_indexer(P: Problem, q_idx, k_idx, w, q_scale=None, k_scale=None, idx=None, vals=None,
                  want_vals: bool = False, ws: Optional[Workspace] = None):
    """Scoring + head weighting + Top-K in one call: (idx, vals or None)."""
    _check_indexer(P, q_idx, k_idx, w, q_scale, k_scale)
    dev = k_idx.device
    idx, vals = _idx_out(P, idx, vals, dev, want_vals)
    ws = _workspace(ws, dev, P.workspace_size(_abi.OP_FUSED_INDEXER))
    _abi.check(lib().dsa_fused_indexer(
        ctypes.byref(P.c), q_idx.data_ptr(), k_idx.data_ptr(), w.data_ptr(), _ptr(q_scale),
        _ptr(k_scale), idx.data_ptr(), _ptr(vals), ws.ptr, ws.nbytes, _stream(dev)))
    return idx, vals


def indexer_prolog(q_proj=None, x=None, w_h=None, q_codes=None, q_scale=None, w=None):
    """Q quantisation and head-weight projection in one launch (dsa_indexer_prolog).

    q_proj [T, H_I, d_I] bf16 -> (q_codes [T, H_I, d_I] uint8 E4M3, q_scale [T, H_I] f32);
    x [T, d_model] bf16, w_h [H_I, d_model] bf16 -> w [T, H_I] f32.  Either part may be
    left out (None inputs).  Returns (q_codes, q_scale, w), None for a part not computed.
    """
    if q_proj is None and x is None:
        raise ValueError("indexer_prolog needs q_proj or (x, w_h)")
    if q_proj is not None:
        T, h, d = q_proj.shape
    else:
        T, h = x.shape[0], w_h.shape[0]
        d = 8
    dev = (q_proj if q_proj is not None else x).device
    d_model = 0
    if q_proj is not None:
        _need(q_proj, "q_proj", _abi.DSA_BF16, (T, h, d))
        if q_codes is None:
            q_codes = torch.empty((T, h, d), dtype=torch.uint8, device=dev)
        if q_scale is None:
            q_scale = torch.empty((T, h), dtype=torch.float32, device=dev)
        _need(q_codes, "q_codes", _abi.DSA_FP8_E4M3, (T, h, d))
        _need(q_scale, "q_scale", _abi.DSA_F32, (T, h))
    else:
        q_codes = q_scale = None
    if x is not None or w_h is not None:
        if x is None or w_h is None:
            raise ValueError("x and w_h go together")
        d_model = x.shape[1]
        _need(x, "x", _abi.DSA_BF16, (T, d_model))
        _need(w_h, "w_h", _abi.DSA_BF16, (h, d_model))
        if w is None:
            w = torch.empty((T, h), dtype=torch.float32, device=dev)
        _need(w, "w", _abi.DSA_F32, (T, h))
    else:
        w = None
    _abi.check(lib().dsa_indexer_prolog(T, h, d, d_model, _ptr(q_proj), _ptr(x), _ptr(w_h),
                                        _ptr(q_codes), _ptr(q_scale), _ptr(w), _stream(dev)))
    return q_codes, q_scale, w


def _attn_out(P: Problem, out, lse, device, want_lse: bool):
    if out is None:
        out = torch.empty(P.total_q, P.h, P.d_c, dtype=_TORCH_OUT[P.out_dtype], device=device)
    _need(out, "out", P.out_dtype, (P.total_q, P.h, P.d_c))
    if lse is None and want_lse:
        lse = torch.empty(P.total_q, P.h, dtype=torch.float32, device=device)
    _need(lse, "lse", _abi.DSA_F32, (P.total_q, P.h), optional=True)
    return out, lse


def sparse_mla_attn(P: Problem, q, kv, idx, out=None, lse=None, want_lse: bool = True,
                    ws: Optional[Workspace] = None):
    """Sparse attention over the latent rows idx selects: (out[ΣT, H, d_c], lse or None)."""
    _need(q, "q", P.kv_dtype, (P.total_q, P.h, P.d))
    _need(kv, "kv", P.kv_dtype, (P.cache_rows, P.d))
    _need(idx, "idx", None, (P.total_q, P.top_k))
    dev = kv.device
    out, lse = _attn_out(P, out, lse, dev, want_lse)
    ws = _workspace(ws, dev, P.workspace_size(_abi.OP_SPARSE_MLA_ATTN))
    _abi.check(lib().dsa_sparse_mla_attn(ctypes.byref(P.c), q.data_ptr(), kv.data_ptr(),
                                         idx.data_ptr(), out.data_ptr(), _ptr(lse), ws.ptr,
                                         ws.nbytes, _stream(dev)))
    return out, lse


def fused_forward(P: Problem, q_idx, k_idx, w, q, kv, q_scale=None, k_scale=None, out=None,
                  lse=None, idx=None, vals=None, want_lse: bool = True, want_idx: bool = True,
                  want_vals: bool = False, ws: Optional[Workspace] = None):
    """The DSA layer: fused indexer then sparse attention → (out, lse, idx, vals)."""
    _check_indexer(P, q_idx, k_idx, w, q_scale, k_scale)
    _need(q, "q", P.kv_dtype, (P.total_q, P.h, P.d))
    _need(kv, "kv", P.kv_dtype, (P.cache_rows, P.d))
    dev = kv.device
    out, lse = _attn_out(P, out, lse, dev, want_lse)
    if want_idx or idx is not None:
        idx, vals = _idx_out(P, idx, vals, dev, want_vals)
    elif want_vals or vals is not None:
        raise ValueError("vals needs idx")
    ws = _workspace(ws, dev, P.workspace_size(_abi.OP_FUSED_FORWARD))
    _abi.check(lib().dsa_fused_forward(
        ctypes.byref(P.c), q_idx.data_ptr(), k_idx.data_ptr(), w.data_ptr(), _ptr(q_scale),
        _ptr(k_scale), q.data_ptr(), kv.data_ptr(), out.data_ptr(), _ptr(lse), _ptr(idx),
        _ptr(vals), ws.ptr, ws.nbytes, _stream(dev)))
    return out, lse, idx, vals


# ---------------------------------------------------------------------------
# Operators around the caches.  Their small calls cost as much on the host as on the GPU, so the
# checks are written out (no objects built, nothing looked up twice).

_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # absent without CUDA: nothing is called then
_current_device = getattr(torch._C, "_cuda_getDevice", None)
_capturing = getattr(torch._C, "_cuda_isCurrentStreamCapturing", None)
_CODES = (torch.uint8, torch.float8_e4m3fn)
_TORCH_DT = {_abi.DSA_F32: (torch.float32,), _abi.DSA_BF16: (torch.bfloat16,),
             _abi.DSA_FP8_E4M3: _CODES}
_F32, _I32, _U8 = (torch.float32,), (torch.int32,), _CODES

_op_ws = threading.local()  # its attributes' dictionary: a thread's workspaces by (device, stream)


def _op_workspace(ws: Optional[Workspace], index: int, stream: int, nbytes: int) -> Workspace:
    """The caller's workspace, grown as needed, or this host thread's own of the device and stream: calls on
    two streams do not share scratch, nor do two threads' calls, whose launches may alternate on one stream.  (A workspace that a
    caller hands to several threads' calls is theirs to take turns with.)  A
    captured call has to bring its workspace: graphs captured on one stream may be replayed on two, and
    memory allocated while capturing would belong to the graph."""
    if ws is not None:
        if ws.buf.get_device() != index:
            raise ValueError(f"the workspace is on {ws.buf.device}, the tensors on cuda:{index}")
        if ws.nbytes < nbytes:
            if _capturing():
                raise ValueError(f"a captured call needs a workspace of {nbytes} bytes beforehand")
            ws.ensure(nbytes)
        return ws
    if _capturing():
        raise ValueError(f"a captured call needs a workspace of its own: ws=Workspace(nbytes={nbytes})")
    mine = _op_ws.__dict__
    held = mine.get((index, stream))
    if held is None or held.nbytes < nbytes:
        size = max(nbytes, 2 * held.nbytes if held else 0)
        held = mine[index, stream] = Workspace(torch.device("cuda", index), size)
    return held


def _want(t, name: str, dtypes, shape, index: int) -> None:
    """A contiguous CUDA tensor of a dtype, shape and device."""
    if t is None:
        raise ValueError(f"{name} is required")
    if t.dtype in dtypes and t.shape == shape and t.get_device() == index and t.is_contiguous():
        return
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} has dtype {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")


def _there(P: Problem, index: int) -> None:
    """A Problem's tensors are on the call's device."""
    if P._device != index:
        raise ValueError(f"the problem's offsets are on cuda:{P._device}, the tensors on cuda:{index}")


def _elsewhere(index: int, f, *args, **kw):
    """A call whose tensors are on another device than the current one: made with that one current."""
    with torch.cuda.device(index):
        return f(*args, **kw)


def _row_stride(t: torch.Tensor, name: str) -> int:
    """Row stride in elements of a tensor [..., d] whose rows are evenly spaced."""
    if t.is_contiguous():
        return t.shape[-1]
    shape, strides = t.shape, t.stride()
    d = shape[-1]
    if d > 1 and strides[-1] != 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    step, n = None, 1
    for size, stride in zip(shape[-2::-1], strides[-2::-1]):
        if size == 1:
            continue
        if step is None:
            step = stride
        elif stride != step * n:
            raise ValueError(f"{name}'s rows must be evenly spaced")
        n *= size
    if step is None:
        return d
    if step < d:
        raise ValueError(f"{name}'s rows overlap")
    return step


def add_rmsnorm(x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None,
                eps: float = 1e-6, quant: Optional[str] = None, want_y: Optional[bool] = None,
                h=None, y=None, codes=None, scale=None):
    """Residual addition and RMS norm, optionally with 8-bit output (dsa_add_rmsnorm).

    x [..., d] (rows evenly spaced, e.g. a slice of a wider projection), residual like x, weight
    [d], all f32 or all bf16.  Returns (y, h, codes, scale): h = x + residual (None without a
    residual; pass h=residual to update it in place), y = the normalised rows (by default where
    quant is None), and for quant "e4m3" codes [..., d] uint8 with scale [...] f32, for "mxfp8"
    codes with E8M0 scale [..., d/32] uint8: on rows of d_idx elements the k_idx and k_scale
    of the indexer.  None for a part not computed.
    """
    if not x.is_cuda:
        raise ValueError("x must be a CUDA tensor")
    dtype, shape, index = x.dtype, x.shape, x.get_device()
    if dtype is torch.bfloat16:
        dt = _abi.DSA_BF16
    elif dtype is torch.float32:
        dt = _abi.DSA_F32
    else:
        raise ValueError(f"x has dtype {dtype}")
    if not shape or shape[-1] < 1:
        raise ValueError("x needs a last dimension of at least 1")
    if index != _current_device():
        return _elsewhere(index, add_rmsnorm, x, weight, residual, eps, quant, want_y, h, y, codes, scale)
    d = shape[-1]
    ld_x = d if x.is_contiguous() else _row_stride(x, "x")
    if weight.dtype is not dtype or weight.shape != (d,) or weight.get_device() != index \
            or not weight.is_contiguous():
        _want(weight, "weight", (dtype,), (d,), index)
    ld_r = res_ptr = h_ptr = y_ptr = codes_ptr = scale_ptr = code = 0
    if residual is not None:
        if residual.dtype != dtype or residual.shape != shape or residual.get_device() != index:
            raise ValueError("residual must have x's shape, dtype and device")
        ld_r = d if residual.is_contiguous() else _row_stride(residual, "residual")
        res_ptr = residual.data_ptr()
        if h is None:
            h = torch.empty(shape, dtype=dtype, device=x.device)
        else:
            _want(h, "h", (dtype,), shape, index)
        h_ptr = h.data_ptr()
    elif h is not None:
        raise ValueError("h needs a residual")
    if y is not None:
        _want(y, "y", (dtype,), shape, index)
        y_ptr = y.data_ptr()
    elif quant is None or want_y:
        y = torch.empty(shape, dtype=dtype, device=x.device)
        y_ptr = y.data_ptr()
    if quant is not None:
        if quant == "mxfp8":
            if d % 32:
                raise ValueError(f"mxfp8 needs a last dimension that is a multiple of 32, not {d}")
            code, sdt, sshape = _abi.DSA_MXFP8_E4M3, torch.uint8, shape[:-1] + (d // 32,)
        elif quant == "e4m3":
            code, sdt, sshape = _abi.DSA_FP8_E4M3, torch.float32, shape[:-1]
        else:
            raise ValueError(f"quant is {quant!r}, expected None, 'e4m3' or 'mxfp8'")
        if codes is None:
            codes = torch.empty(shape, dtype=torch.uint8, device=x.device)
        else:
            _want(codes, "codes", _CODES, shape, index)
        if scale is None:
            scale = torch.empty(sshape, dtype=sdt, device=x.device)
        else:
            _want(scale, "scale", (sdt,), sshape, index)
        codes_ptr, scale_ptr = codes.data_ptr(), scale.data_ptr()
    elif codes is not None or scale is not None:
        raise ValueError("codes and scale need quant")
    rc = lib().dsa_add_rmsnorm(x.numel() // d, d, dt, code, eps, x.data_ptr(), ld_x, res_ptr, ld_r,
                               weight.data_ptr(), h_ptr, y_ptr, codes_ptr, scale_ptr,
                               _raw_stream(index))
    if rc:
        _abi.check(rc)
    return y, h, codes, scale


def _ws_bytes(P: Problem, op: int) -> int:
    """P's workspace size for an op (on P's device, which is current), asked for once."""
    n = P._ws_sizes.get(op)
    if n is None:
        n = P._ws_sizes[op] = P.workspace_size(op)
    return n


def prefix_mla_attn(P: Problem, q, kv, prefix_kv=None, prefix_table=None,
                    prefix_len: Optional[int] = None, out=None, lse=None, want_lse: bool = True,
                    ws: Optional[Workspace] = None):
    """Dense MLA attention of all sequences over one shared prefix and, causally, over their own
    latent rows (dsa_prefix_mla_attn): (out[ΣT, H, d_c], lse or None).

    P describes the sequences behind the prefix.  The prefix is prefix_kv [prefix_len, D], or, in a
    paged cache, the pages prefix_table [>= ceil(prefix_len / page_size)] int32 of kv; without
    either there is none.  A captured call needs ws."""
    if not kv.is_cuda:
        raise ValueError("kv must be a CUDA tensor")
    index, dts = kv.get_device(), _TORCH_DT[P.kv_dtype]
    if index != _current_device():
        return _elsewhere(index, prefix_mla_attn, P, q, kv, prefix_kv, prefix_table, prefix_len, out, lse,
                          want_lse, ws)
    q_shape, kv_shape, out_shape, lse_shape, _ = P._shapes
    _want(q, "q", dts, q_shape, index)
    _want(kv, "kv", dts, kv_shape, index)
    _there(P, index)
    n = pre_ptr = table_ptr = 0
    if prefix_kv is not None:
        if prefix_table is not None:
            raise ValueError("prefix_kv and prefix_table exclude each other")
        if prefix_kv.dim() != 2:
            raise ValueError(f"prefix_kv has shape {tuple(prefix_kv.shape)}")
        rows = prefix_kv.shape[0]
        _want(prefix_kv, "prefix_kv", dts, (rows, kv_shape[1]), index)
        n = rows if prefix_len is None else int(prefix_len)
        if not 0 <= n <= rows:
            raise ValueError(f"prefix_len is {n}, prefix_kv has {rows} rows")
        pre_ptr = prefix_kv.data_ptr() if n else 0
    elif prefix_table is not None:
        if not P.page_size:
            raise ValueError("prefix_table needs paged caches")
        if prefix_len is None:
            raise ValueError("prefix_table needs prefix_len")
        n = int(prefix_len)
        if prefix_table.dim() != 1 or n < 0 or prefix_table.numel() * P.page_size < n:
            raise ValueError("prefix_table must be an int32 tensor [pages] that covers prefix_len")
        _want(prefix_table, "prefix_table", _I32, prefix_table.shape, index)
        table_ptr = prefix_table.data_ptr() if n else 0
    elif prefix_len:
        raise ValueError("prefix_len needs prefix_kv or prefix_table")
    if out is None:
        out = torch.empty(out_shape, dtype=_TORCH_OUT[P.out_dtype], device=kv.device)
    else:
        _want(out, "out", _TORCH_DT[P.out_dtype], out_shape, index)
    if lse is not None:
        _want(lse, "lse", _F32, lse_shape, index)
    elif want_lse:
        lse = torch.empty(lse_shape, dtype=torch.float32, device=kv.device)
    stream = _raw_stream(index)
    ws = _op_workspace(ws, index, stream, _ws_bytes(P, _abi.OP_PREFIX_MLA_ATTN))
    rc = lib().dsa_prefix_mla_attn(P._ref, n, pre_ptr, table_ptr, q.data_ptr(), kv.data_ptr(),
                                   out.data_ptr(), 0 if lse is None else lse.data_ptr(),
                                   ws.buf.data_ptr(), ws.nbytes, stream)
    if rc:
        _abi.check(rc)
    return out, lse


def accumulate_attn_weights(P: Problem, q, kv, idx, lse, acc, ws: Optional[Workspace] = None):
    """Add the attention weight every selected position received, summed over heads and queries,
    to acc [B, >= max_k_len] f32 in place (dsa_accumulate_attn_weights); returns acc.  idx and lse
    are those of sparse_mla_attn or fused_forward on the same q and kv.  A captured call needs ws."""
    if not kv.is_cuda:
        raise ValueError("kv must be a CUDA tensor")
    index, dts = kv.get_device(), _TORCH_DT[P.kv_dtype]
    if index != _current_device():
        return _elsewhere(index, accumulate_attn_weights, P, q, kv, idx, lse, acc, ws)
    q_shape, kv_shape, _, lse_shape, idx_shape = P._shapes
    _want(q, "q", dts, q_shape, index)
    _want(kv, "kv", dts, kv_shape, index)
    _want(idx, "idx", _I32, idx_shape, index)
    _want(lse, "lse", _F32, lse_shape, index)
    ld = _acc_stride(P, acc, "acc", P.max_k_len, index)
    _there(P, index)
    stream = _raw_stream(index)
    ws = _op_workspace(ws, index, stream, _ws_bytes(P, _abi.OP_ATTN_WEIGHTS))
    rc = lib().dsa_accumulate_attn_weights(P._ref, q.data_ptr(), kv.data_ptr(), idx.data_ptr(),
                                           lse.data_ptr(), acc.data_ptr(), ld, ws.buf.data_ptr(),
                                           ws.nbytes, stream)
    if rc:
        _abi.check(rc)
    return acc


def _acc_stride(P: Problem, acc, name: str, width: int, index: int) -> int:
    """Row stride of an accumulator [B, >= width] f32 (rows contiguous, any stride between)."""
    B = P.c.num_seqs
    if acc.dtype is not torch.float32 or acc.dim() != 2 or acc.get_device() != index \
            or acc.shape[0] != B or acc.shape[1] < width \
            or not (acc.is_contiguous() or ((acc.shape[1] == 1 or acc.stride(1) == 1)
                                            and (B == 1 or acc.stride(0) >= acc.shape[1]))):
        raise ValueError(f"{name} must be a float32 tensor [{B}, >= {width}] on cuda:{index} with "
                         "contiguous rows")
    return acc.stride(0) if B > 1 else acc.shape[1]


class Eviction(NamedTuple):
    """What evict() kept: kept [B, budget] int32 (-1 padded), cu_k [B+1] int32 and k_lens (host) of
    the smaller caches, acc [B, budget] f32, and the caches' moved tensors (None: not moved)."""

    kept: torch.Tensor
    cu_k: torch.Tensor
    k_lens: list
    acc: Optional[torch.Tensor]
    kv: Optional[torch.Tensor]
    k_idx: Optional[torch.Tensor]
    k_scale: Optional[torch.Tensor]


def evict(P: Problem, acc, budget: int, sink: int = 0, recent: int = 0, kv=None, k_idx=None,
          k_scale=None, kv_out=None, k_idx_out=None, k_scale_out=None, block_table_out=None,
          kept=None, cu_k_out=None, acc_out=None, ws: Optional[Workspace] = None) -> Eviction:
    """Keep each sequence's first `sink`, last `recent` and, by acc, best other positions, `budget`
    in all, and move their cache rows (dsa_evict).

    The destination is packed (kv_out, k_idx_out, k_scale_out with at least sum(k_lens) rows of
    the result; allocated where None) or, with block_table_out [B, pages] int32, paged with P's
    page size (the *_out tensors are then required; they may be the source's pool, on other pages).
    acc_out [B, >= budget] receives the kept positions' acc and zeros behind them up to column
    budget.  A captured call needs ws."""
    if not acc.is_cuda:
        raise ValueError("acc must be a CUDA tensor")
    if acc.get_device() != _current_device():
        return _elsewhere(acc.get_device(), evict, P, acc, budget, sink, recent, kv, k_idx, k_scale, kv_out,
                          k_idx_out, k_scale_out, block_table_out, kept, cu_k_out, acc_out, ws)
    budget, sink, recent, table = int(budget), int(sink), int(recent), block_table_out
    src, dst = (kv, k_idx, k_scale), (kv_out, k_idx_out, k_scale_out)
    if budget < 1 or sink < 0 or recent < 0 or sink + recent > budget:
        raise ValueError(f"budget = {budget}, sink = {sink}, recent = {recent}: 1 <= budget and "
                         "sink + recent <= budget are needed")
    B, dev, index = P.c.num_seqs, acc.device, acc.get_device()
    ld = _acc_stride(P, acc, "acc", P.max_k_len, index)
    _there(P, index)
    k_lens = [n if n < budget else budget for n in P.k_lens]
    rows = sum(k_lens)
    max_pages = num_pages = table_ptr = 0
    if table is not None:
        if not P.page_size:
            raise ValueError("block_table_out needs paged caches")
        if table.dim() != 2 or table.shape[0] != B or table.shape[1] * P.page_size < max(k_lens):
            raise ValueError("block_table_out must be an int32 tensor [B, pages] that covers the kept "
                             "positions")
        _want(table, "block_table_out", _I32, table.shape, index)
        max_pages, table_ptr = table.shape[1], table.data_ptr()
    specs = P._row_specs
    if specs is None:  # of a row of each cache: name, dtypes, shape of the cache, shape of a row
        mx, n = P.idx_dtype == _abi.DSA_MXFP8_E4M3, P.cache_rows
        tails = ((P.d,), (P.d_idx,), (P.d_idx // 32,) if mx else ())
        dts = (_TORCH_DT[P.kv_dtype], _CODES if mx else _TORCH_DT[P.idx_dtype], _U8 if mx else _F32)
        specs = P._row_specs = tuple((name, dt, (n,) + tail, tail) for name, dt, tail in
                                     zip(("kv", "k_idx", "k_scale"), dts, tails))
    if k_scale is not None and P.idx_dtype not in (_abi.DSA_FP8_E4M3, _abi.DSA_MXFP8_E4M3):
        raise ValueError("k_scale goes with FP8 or MXFP8 index keys")
    moved, ptrs, rows_out = [], [], None
    for s, o, (name, dts, whole, tail) in zip(src, dst, specs):
        if s is None:
            if o is not None:
                raise ValueError(f"{name}_out needs {name}")
            moved.append(None)
            ptrs += (0, 0)
            continue
        _want(s, name, dts, whole, index)
        if o is None:
            if table is not None:
                raise ValueError(f"a paged destination needs {name}_out")
            o = torch.empty((rows,) + tail, dtype=s.dtype, device=dev)
        elif o.dim() != 1 + len(tail):
            raise ValueError(f"{name}_out has shape {tuple(o.shape)}")
        else:
            _want(o, name + "_out", dts, (o.shape[0],) + tail, index)
        n = o.shape[0]
        if n < rows or (rows_out is not None and n != rows_out) or (table is not None and n % P.page_size):
            raise ValueError(f"{name}_out has {n} rows: all destinations need the same number, at "
                             f"least {rows}, whole pages where they are paged")
        rows_out = n
        moved.append(o)
        ptrs += (s.data_ptr(), o.data_ptr())
    if table is not None:
        num_pages = (P.cache_rows if rows_out is None else rows_out) // P.page_size
    if kept is None:
        kept = torch.empty((B, budget), dtype=torch.int32, device=dev)
    else:
        _want(kept, "kept", _I32, (B, budget), index)
    if cu_k_out is None:
        cu_k_out = torch.empty((B + 1,), dtype=torch.int32, device=dev)
    else:
        _want(cu_k_out, "cu_k_out", _I32, (B + 1,), index)
    if acc_out is None:
        acc_out, ld_out = torch.empty((B, budget), dtype=torch.float32, device=dev), budget
    else:
        ld_out = _acc_stride(P, acc_out, "acc_out", budget, index)
    stream = _raw_stream(index)
    ws = _op_workspace(ws, index, stream, _ws_bytes(P, _abi.OP_EVICT))
    rc = lib().dsa_evict(P._ref, acc.data_ptr(), ld, budget, sink, recent, kept.data_ptr(),
                         cu_k_out.data_ptr(), acc_out.data_ptr(), ld_out, *ptrs, table_ptr, max_pages,
                         num_pages, rows_out or 0, ws.buf.data_ptr(), ws.nbytes, stream)
    if rc:
        _abi.check(rc)
    return Eviction(kept, cu_k_out, k_lens, acc_out, *moved)


# ---------------------------------------------------------------------------
# The latent cache in 4 bits, rotary positions and pages.

class Rotary:
    """Frequencies and axes of a rotation of d_rope columns: pair i turns by inv_freq[i] radians a position of its axis.

    sections: pairs of each axis in order, d_rope / 2 together (default: one axis); or axes: the axis of
    every pair.  inv_freq: d_rope / 2 frequencies (default theta ** (-2 i / d_rope)).  interleaved: pair i is columns 2i and
    2i + 1, otherwise i and i + d_rope / 2.  Host data only: one object serves every device and stream."""

    def __init__(self, d_rope: int, sections: Optional[Sequence[int]] = None, theta: float = 10000.0,
                 inv_freq: Optional[Sequence[float]] = None, axes: Optional[Sequence[int]] = None,
                 interleaved: bool = True):
        if d_rope < 2 or d_rope % 2 or d_rope > 256:
            raise ValueError(f"d_rope is {d_rope}: an even number from 2 to 256 is needed")
        n = d_rope // 2
        if inv_freq is None:
            inv_freq = [float(theta) ** (-i / n) for i in range(n)]
        inv_freq = [float(f) for f in inv_freq]
        if sections is not None:
            if axes is not None:
                raise ValueError("sections and axes exclude each other")
            if any(k < 0 for k in sections):
                raise ValueError("sections must not be negative")
            axes, num = [a for a, k in enumerate(sections) for _ in range(k)], len(sections)
        else:
            axes = [0] * n if axes is None else [int(a) for a in axes]
            num = max(axes, default=0) + 1
        if len(inv_freq) != n or len(axes) != n:
            raise ValueError(f"{n} pairs need {n} frequencies and axes, not {len(inv_freq)} and {len(axes)}")
        if not all(math.isfinite(f) for f in inv_freq) or min(axes) < 0 or not 1 <= num <= 255:
            raise ValueError("frequencies must be finite, axes from 0 to 254")
        self.d_rope, self.num_axes, self.interleaved = d_rope, num, bool(interleaved)
        # turns a position as a fraction of 2^64 (of the 64-bit quotient, exactly)
        self.turn = (ctypes.c_uint64 * n)(*(_turn(f) for f in inv_freq))
        self.axis = (ctypes.c_uint8 * n)(*axes)


def _turn(f: float) -> int:
    num, den = (f / (2.0 * math.pi)).as_integer_ratio()
    return ((num << 65) // den + 1 >> 1) % (1 << 64)


def _head_strides(t: torch.Tensor, name: str, d: int):
    """(tokens, heads, token stride, head stride) of a tensor [T, H, d] or [T, d] with contiguous columns."""
    if t.dim() == 2:
        (T, c), (st, sc) = t.shape, t.stride()
        H, sh = 1, d
    elif t.dim() == 3:
        (T, H, c), (st, sh, sc) = t.shape, t.stride()
    else:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected [T, H, {d}] or [T, {d}]")
    if c != d:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {d} columns")
    if sc != 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    return T, H, st, sh


def rotate_axes(x: torch.Tensor, positions: torch.Tensor, rotary: Rotary, out=None, inverse: bool = False):
    """Rotate rope columns x [T, H, d_rope] or [T, d_rope] (f32 or bf16, any strides of tokens and heads, e.g. the
    last columns of the queries) by positions [axes, T] or, with one axis, [T] int32 (dsa_rotate_axes).

    out: like x, its own strides; out=x rotates in place; a new contiguous tensor by default.  inverse turns
    back.  Returns out."""
    if not x.is_cuda:
        raise ValueError("x must be a CUDA tensor")
    dtype, index, d = x.dtype, x.get_device(), rotary.d_rope
    if dtype is torch.bfloat16:
        dt = _abi.DSA_BF16
    elif dtype is torch.float32:
        dt = _abi.DSA_F32
    else:
        raise ValueError(f"x has dtype {dtype}")
    if index != _current_device():
        return _elsewhere(index, rotate_axes, x, positions, rotary, out, inverse)
    T, H, st, sh = _head_strides(x, "x", d)
    if positions.dtype is not torch.int32 or positions.get_device() != index:
        raise ValueError(f"positions must be an int32 tensor on cuda:{index}")
    shape, n = positions.shape, rotary.num_axes
    if shape != (n, T) and not (n == 1 and shape == (T,)):
        raise ValueError(f"positions has shape {tuple(shape)}, expected {(n, T)}")
    if T > 1 and positions.stride(-1) != 1:
        raise ValueError("positions' last dimension must be contiguous")
    ld = positions.stride(0) if n > 1 else T
    if out is None:
        out = torch.empty(x.shape, dtype=dtype, device=x.device)
    elif out.dtype is not dtype or out.shape != x.shape or out.get_device() != index:
        raise ValueError("out must have x's shape, dtype and device")
    if H == 0:
        return out
    _, _, ot, oh = _head_strides(out, "out", d)
    rc = lib().dsa_rotate_axes(T, H, d, dt, rotary.interleaved, bool(inverse), n, rotary.turn, rotary.axis,
                               positions.data_ptr(), ld, x.data_ptr(), st, sh, out.data_ptr(), ot, oh,
                               _raw_stream(index))
    if rc:
        _abi.check(rc)
    return out


def kv4_row_bytes(d_c: int, d_rope: int) -> int:
    """Bytes of a row of the 4-bit latent cache (512 + 64 columns: 416)."""
    n = ctypes.c_int32(0)
    _abi.check(lib().dsa_kv4_row_bytes(d_c, d_rope, ctypes.byref(n)))
    return n.value


def _kv4_shape(P: Problem):
    shape = P.__dict__.get("_kv4")
    if shape is None:
        shape = P._kv4 = (P.cache_rows, kv4_row_bytes(P.d_c, P.d_rope))
    return shape


def _row_tensor(t, name: str, dts, rows: int, width: int, index: int) -> int:
    """Row stride of a tensor [rows, width] with contiguous rows."""
    if t is None or t.dtype not in dts or t.get_device() != index or t.shape != (rows, width):
        raise ValueError(f"{name} must be a {dts[0]} tensor {[rows, width]} on cuda:{index}")
    return width if t.is_contiguous() else _row_stride(t, name)


def write_kv4(P: Problem, latent, k_rope, kv4, ws: Optional[Workspace] = None):
    """Write the rows of P's new tokens (the last of each sequence) to the 4-bit latent cache (dsa_write_kv4).

    latent [total_q, d_c] and k_rope [total_q, d_rope] (None without rope columns) of P's kv_dtype, e.g. slices of a
    projection's output; kv4 [cache rows, kv4_row_bytes(d_c, d_rope)] uint8.  Returns kv4.  A captured call needs ws."""
    if not kv4.is_cuda:
        raise ValueError("kv4 must be a CUDA tensor")
    index, dts = kv4.get_device(), _TORCH_DT[P.kv_dtype]
    if index != _current_device():
        return _elsewhere(index, write_kv4, P, latent, k_rope, kv4, ws)
    _want(kv4, "kv4", (torch.uint8,), _kv4_shape(P), index)
    _there(P, index)
    ld = _row_tensor(latent, "latent", dts, P.c.total_q, P.d_c, index)
    rope = ld_rope = 0
    if P.d_rope:
        ld_rope = _row_tensor(k_rope, "k_rope", dts, P.c.total_q, P.d_rope, index)
        rope = k_rope.data_ptr()
    stream = _raw_stream(index)
    ws = _op_workspace(ws, index, stream, STATUS_BYTES)
    rc = lib().dsa_write_kv4(P._ref, latent.data_ptr(), ld, rope, ld_rope, kv4.data_ptr(), ws.buf.data_ptr(), ws.nbytes,
                             stream)
    if rc:
        _abi.check(rc)
    return kv4


def read_kv4(P: Problem, kv4, out=None, ws: Optional[Workspace] = None):
    """Every position's row of the 4-bit latent cache, decoded and packed: out [total_k, D] of P's kv_dtype
    (dsa_read_kv4).  A captured call needs ws."""
    if not kv4.is_cuda:
        raise ValueError("kv4 must be a CUDA tensor")
    index = kv4.get_device()
    if index != _current_device():
        return _elsewhere(index, read_kv4, P, kv4, out, ws)
    _want(kv4, "kv4", (torch.uint8,), _kv4_shape(P), index)
    _there(P, index)
    if out is None:
        out = torch.empty((P.c.total_k, P.d), dtype=_TORCH_OUT[P.kv_dtype], device=kv4.device)
    else:
        _want(out, "out", _TORCH_DT[P.kv_dtype], (P.c.total_k, P.d), index)
    stream = _raw_stream(index)
    ws = _op_workspace(ws, index, stream, STATUS_BYTES)
    rc = lib().dsa_read_kv4(P._ref, kv4.data_ptr(), out.data_ptr(), ws.buf.data_ptr(), ws.nbytes, stream)
    if rc:
        _abi.check(rc)
    return out


def sparse_mla_attn4(P: Problem, q, kv4, idx, out=None, lse=None, want_lse: bool = True,
                     ws: Optional[Workspace] = None):
    """sparse_mla_attn over the 4-bit latent cache kv4 [cache rows, kv4_row_bytes(d_c, d_rope)] uint8
    (dsa_sparse_mla_attn4): (out[ΣT, H, d_c], lse or None).  A captured call needs ws.

    With bf16 queries over 512 + 64 columns probabilities are rounded to bf16 (also for f32 outputs), and a head's latent query
    columns are exact down to 2^-29 of its largest one and 0 below 2^-39 of it."""
    if not kv4.is_cuda:
        raise ValueError("kv4 must be a CUDA tensor")
    index = kv4.get_device()
    if index != _current_device():
        return _elsewhere(index, sparse_mla_attn4, P, q, kv4, idx, out, lse, want_lse, ws)
    q_shape, _, out_shape, lse_shape, idx_shape = P._shapes
    _want(q, "q", _TORCH_DT[P.kv_dtype], q_shape, index)
    _want(kv4, "kv4", (torch.uint8,), _kv4_shape(P), index)
    _want(idx, "idx", _I32, idx_shape, index)
    _there(P, index)
    if out is None:
        out = torch.empty(out_shape, dtype=_TORCH_OUT[P.out_dtype], device=kv4.device)
    else:
        _want(out, "out", _TORCH_DT[P.out_dtype], out_shape, index)
    if lse is not None:
        _want(lse, "lse", _F32, lse_shape, index)
    elif want_lse:
        lse = torch.empty(lse_shape, dtype=torch.float32, device=kv4.device)
    stream = _raw_stream(index)
    ws = _op_workspace(ws, index, stream, _ws_bytes(P, _abi.OP_SPARSE_MLA_ATTN4))
    rc = lib().dsa_sparse_mla_attn4(P._ref, q.data_ptr(), kv4.data_ptr(), idx.data_ptr(), out.data_ptr(),
                                    0 if lse is None else lse.data_ptr(), ws.buf.data_ptr(), ws.nbytes, stream)
    if rc:
        _abi.check(rc)
    return out, lse


def _pages_of(table, refs, index: int):
    """(address, rows, width, row stride) of a block table [rows, width] int32; refs [pages] int32."""
    if table.dtype is not torch.int32 or table.dim() != 2 or 0 in table.shape \
            or not (table.is_contiguous() or ((table.shape[1] == 1 or table.stride(1) == 1)
                                              and (table.shape[0] == 1 or table.stride(0) >= table.shape[1]))):
        raise ValueError("table must be an int32 tensor [rows, pages] with contiguous rows")
    if refs.dtype is not torch.int32 or refs.dim() != 1 or refs.get_device() != index or not refs.is_contiguous() \
            or not refs.numel():
        raise ValueError(f"refs must be a contiguous int32 tensor [num_pages] on cuda:{index}")
    rows, width = table.shape
    return table.data_ptr(), rows, width, table.stride(0) if rows > 1 else width


def _entries(named, index: int) -> int:
    """Number of entries of index tensors [n] int32."""
    n = None
    for name, t in named:
        if t.dtype is not torch.int32 or t.dim() != 1 or t.get_device() != index or not t.is_contiguous() \
                or (n is not None and t.shape[0] != n):
            raise ValueError(f"{name} must be a contiguous int32 tensor [{'n' if n is None else n}] on cuda:{index}")
        n = t.shape[0]
    return n


def _cache_list(caches, rows: int, index: int):
    """(number, their addresses, their row bytes) of caches with `rows` rows: one array, kept by the caller while its
    address is in use."""
    at, size = [], []
    for t in caches:
        shape = t.shape
        if not shape or shape[0] != rows or t.get_device() != index or not t.is_contiguous():
            raise ValueError(f"caches[{len(at)}] must be a contiguous tensor of {rows} rows on cuda:{index}")
        at.append(t.data_ptr())
        size.append(t.nbytes // rows)
    return len(at), array.array("q", at + size)


_page_ws = {}  # workspace bytes by (rows, entries, pages)


def _pages_ws(ws, index: int, stream: int, rows: int, n: int, pages: int) -> Workspace:
    key = (rows, n, pages)
    size = _page_ws.get(key)
    if size is None:
        b = ctypes.c_size_t(0)
        _abi.check(lib().dsa_pages_workspace_size(rows, n, pages, ctypes.byref(b)))
        if len(_page_ws) > 4096:
            _page_ws.clear()
        size = _page_ws[key] = b.value
    return _op_workspace(ws, index, stream, size)


def fork_pages(table, refs, src, dst, lens, page_size: int, ws: Optional[Workspace] = None):
    """Row dst[i] of the block table gets the pages of row src[i]'s first lens[i] positions, shared (dsa_fork_pages).

    table [rows, pages] int32 (-1 behind a row's pages), refs [num_pages] int32: table entries that hold a page; src, dst,
    lens [n] int32, all on one device.  What dst held is not given back: free_pages first.  reserve_pages then
    makes room for the tokens that follow.  Returns table.  A captured call needs ws."""
    if not table.is_cuda:
        raise ValueError("table must be a CUDA tensor")
    index = table.get_device()
    if index != _current_device():
        return _elsewhere(index, fork_pages, table, refs, src, dst, lens, page_size, ws)
    at, rows, width, ld = _pages_of(table, refs, index)
    n = _entries((("src", src), ("dst", dst), ("lens", lens)), index)
    stream = _raw_stream(index)
    ws = _op_workspace(ws, index, stream, STATUS_BYTES)
    rc = lib().dsa_fork_pages(at, rows, width, ld, refs.data_ptr(), refs.shape[0], page_size, n, src.data_ptr(),
                              dst.data_ptr(), lens.data_ptr(), ws.buf.data_ptr(), ws.nbytes, stream)
    if rc:
        _abi.check(rc)
    return table


def free_pages(table, refs, rows, ws: Optional[Workspace] = None):
    """Give back the pages of the block table's rows named in rows [n] int32 (dsa_free_pages); their entries become
    -1.  Returns table.  A captured call needs ws."""
    if not table.is_cuda:
        raise ValueError("table must be a CUDA tensor")
    index = table.get_device()
    if index != _current_device():
        return _elsewhere(index, free_pages, table, refs, rows, ws)
    at, num, width, ld = _pages_of(table, refs, index)
    n = _entries((("rows", rows),), index)
    stream = _raw_stream(index)
    ws = _op_workspace(ws, index, stream, STATUS_BYTES)
    rc = lib().dsa_free_pages(at, num, width, ld, refs.data_ptr(), refs.shape[0], n, rows.data_ptr(), ws.buf.data_ptr(),
                              ws.nbytes, stream)
    if rc:
        _abi.check(rc)
    return table


def reserve_pages(table, refs, rows, lens, new_lens, page_size: int, caches=(), held=None,
                  ws: Optional[Workspace] = None):
    """Give row rows[i] of the block table, which holds lens[i] positions, pages of its own to write positions lens[i] ..
    new_lens[i] - 1 to (dsa_reserve_pages): new ones, and a copy, in all caches, of a last page that others hold too.

    caches: up to 8 contiguous tensors of num_pages * page_size rows.  Returns held [n] int32: new_lens[i], or lens[i] where
    the free pages did not suffice, for the entry or for another one that shares its last page (ws.status() then has
    DSA_FLAG_NO_PAGES).  A captured call needs ws."""
    if not table.is_cuda:
        raise ValueError("table must be a CUDA tensor")
    index = table.get_device()
    if index != _current_device():
        return _elsewhere(index, reserve_pages, table, refs, rows, lens, new_lens, page_size, caches, held, ws)
    at, num, width, ld = _pages_of(table, refs, index)
    n = _entries((("rows", rows), ("lens", lens), ("new_lens", new_lens)), index)
    count, listed = _cache_list(caches, refs.shape[0] * page_size, index)
    if held is None:
        held = torch.empty((n,), dtype=torch.int32, device=table.device)
    else:
        _want(held, "held", _I32, (n,), index)
    listed_at = listed.buffer_info()[0]
    stream = _raw_stream(index)
    ws = _pages_ws(ws, index, stream, num, n, refs.shape[0])
    rc = lib().dsa_reserve_pages(at, num, width, ld, refs.data_ptr(), refs.shape[0], page_size, n, rows.data_ptr(),
                                 lens.data_ptr(), new_lens.data_ptr(), held.data_ptr(), count, listed_at, listed_at + 8 * count,
                                 ws.buf.data_ptr(), ws.nbytes, stream)
    if rc:
        _abi.check(rc)
    return held


def compact_pages(table, refs, page_size: int, caches=(), moved=None, live=None, ws: Optional[Workspace] = None):
    """Move the pages in use to the front of the pool, in all caches; table and refs follow (dsa_compact_pages).

    Every holder of a page has to be in the table.  Returns (moved [num_pages] int32: where each page went, -1 for a free one;
    live [1] int32: the pages in use).  A captured call needs ws."""
    if not table.is_cuda:
        raise ValueError("table must be a CUDA tensor")
    index = table.get_device()
    if index != _current_device():
        return _elsewhere(index, compact_pages, table, refs, page_size, caches, moved, live, ws)
    at, num, width, ld = _pages_of(table, refs, index)
    pages = refs.shape[0]
    count, listed = _cache_list(caches, pages * page_size, index)
    if moved is None:
        moved = torch.empty((pages,), dtype=torch.int32, device=table.device)
    else:
        _want(moved, "moved", _I32, (pages,), index)
    if live is None:
        live = torch.empty((1,), dtype=torch.int32, device=table.device)
    else:
        _want(live, "live", _I32, (1,), index)
    listed_at = listed.buffer_info()[0]
    stream = _raw_stream(index)
    ws = _pages_ws(ws, index, stream, num, 0, pages)
    rc = lib().dsa_compact_pages(at, num, width, ld, refs.data_ptr(), pages, page_size, moved.data_ptr(), live.data_ptr(),
                                 count, listed_at, listed_at + 8 * count, ws.buf.data_ptr(), ws.nbytes, stream)
    if rc:
        _abi.check(rc)
    return moved, live


class trace:
    """Context manager recording per-launch CUDA-event times of the library's kernels."""

    def __init__(self, capacity: int = 4096):
        self.capacity = capacity
        self.records = []

    def __enter__(self):
        _abi.check(lib().dsa_trace_begin(self.capacity))
        return self

    def __exit__(self, *exc):
        _abi.check(lib().dsa_trace_end())
        n = lib().dsa_trace_count()
        name = ctypes.create_string_buffer(128)
        ms = ctypes.c_float(0)
        self.records = []
        for i in range(n):
            _abi.check(lib().dsa_trace_get(i, name, 128, ctypes.byref(ms)))
            self.records.append((name.value.decode(), ms.value))
        return False
