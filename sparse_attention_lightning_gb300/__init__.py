"""GB300 (sm_103a) DSA hot path: Lightning Indexer → Top-K → sparse MLA attention.

A thin binding over libdsa.so (include/dsa.h).  Functions take CUDA tensors,
check their dtypes and shapes, and pass raw pointers plus the current CUDA
stream to the library; every step of the computation runs in the library's
kernels.  There is no CPU or framework fallback: if the library is missing,
calls raise.

Names follow the C ABI: indexer_scores, topk, fused_indexer, sparse_mla_attn,
fused_forward, indexer_prolog, add_rmsnorm, prefix_mla_attn, accumulate_attn_weights, evict.
"""
from __future__ import annotations

import ctypes
import math
import threading
from typing import NamedTuple, Optional, Sequence, Tuple

import torch

from . import _abi
from ._abi import STATUS_BYTES, DsaError, lib  # noqa: F401

__all__ = ["Problem", "Workspace", "indexer_scores", "topk", "fused_indexer", "sparse_mla_attn",
           "fused_forward", "indexer_prolog", "add_rmsnorm", "prefix_mla_attn",
           "accumulate_attn_weights", "evict", "Eviction", "DsaError", "lib", "trace"]

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
        sequence b is row block_table[b, s // page_size] * page_size + s % page_size."""
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
