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
    word and the kernels' synchronisation counters, zero between calls)."""

    def __init__(self, device=None, nbytes: int = STATUS_BYTES):
        self.device = torch.device(device or "cuda")
        self.buf = torch.zeros(max(STATUS_BYTES, nbytes), dtype=torch.uint8, device=self.device)

    def ensure(self, nbytes: int) -> "Workspace":
        if self.buf.numel() < nbytes:
            flags = self.buf[:STATUS_BYTES].clone()
            self.buf = torch.zeros(nbytes, dtype=torch.uint8, device=self.device)
            self.buf[:STATUS_BYTES].copy_(flags)
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
# Operators around the caches.

_op_ws = {}


def _op_workspace(ws: Optional[Workspace], device: torch.device, nbytes: int) -> Workspace:
    """The caller's workspace, grown as needed, or this device's and stream's own: calls on two
    streams do not share scratch.  A default workspace that grows keeps its earlier buffers
    alive, so a captured graph that refers to one stays valid; while a stream is being captured none
    is allocated (its memory would belong to the graph)."""
    if ws is not None:
        if ws.device.type != device.type or ws.buf.device != device:
            raise ValueError(f"the workspace is on {ws.buf.device}, the tensors on {device}")
        if ws.nbytes < nbytes and torch.cuda.is_current_stream_capturing():
            raise ValueError(f"a captured call needs a workspace of {nbytes} bytes beforehand")
        return ws.ensure(nbytes)
    key = (device.index, _stream(device))
    held = _op_ws.setdefault(key, [])
    if not held or held[-1].nbytes < nbytes:
        if torch.cuda.is_current_stream_capturing():
            raise ValueError("a captured call needs its workspace beforehand: pass ws, or make the "
                             "call once on this stream before capturing it")
        grown = max(nbytes, 2 * held[-1].nbytes if held else 0)
        held.append(Workspace(device, grown))
    return held[-1]


def _same_device(dev: torch.device, **tensors) -> None:
    for name, t in tensors.items():
        if t is not None and t.device != dev:
            raise ValueError(f"{name} is on {t.device}, expected {dev}")


class _on:
    """Makes a device current for a launch (nothing to do where it is already)."""

    __slots__ = ("dev", "prev")

    def __init__(self, dev: torch.device):
        self.dev = dev

    def __enter__(self):
        self.prev = torch.cuda.current_device()
        if self.prev != self.dev.index:
            torch.cuda.set_device(self.dev)

    def __exit__(self, *exc):
        if self.prev != self.dev.index:
            torch.cuda.set_device(self.prev)
        return False


def _rows_2d(t: torch.Tensor, name: str) -> Tuple[int, int]:
    """(rows, row stride in elements) of a tensor [..., d] whose rows are evenly spaced."""
    d = t.shape[-1]
    if d > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    rows = t.numel() // d if d else 0
    if t.dim() == 1 or rows <= 1:
        return rows, d
    step, n = None, 1
    for size, stride in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if size == 1:
            continue
        if step is None:
            step = stride
        elif stride != step * n:
            raise ValueError(f"{name}'s rows must be evenly spaced")
        n *= size
    if step < d:
        raise ValueError(f"{name}'s rows overlap")
    return rows, step


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
    if quant not in (None, "e4m3", "mxfp8"):
        raise ValueError(f"quant is {quant!r}, expected None, 'e4m3' or 'mxfp8'")
    if not x.is_cuda:
        raise ValueError("x must be a CUDA tensor")
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError("x needs a last dimension of at least 1")
    dt = _DT.get(x.dtype)
    if dt not in (_abi.DSA_F32, _abi.DSA_BF16):
        raise ValueError(f"x has dtype {x.dtype}")
    shape, d, dev = tuple(x.shape), x.shape[-1], x.device
    rows, ld_x = _rows_2d(x, "x")
    _need(weight, "weight", dt, (d,))
    ld_r = 0
    if residual is not None:
        if residual.dtype != x.dtype or residual.shape != x.shape or not residual.is_cuda:
            raise ValueError("residual must have x's shape, dtype and device")
        ld_r = _rows_2d(residual, "residual")[1]
        if h is None:
            h = torch.empty(shape, dtype=x.dtype, device=dev)
        _need(h, "h", dt, shape)
    elif h is not None:
        raise ValueError("h needs a residual")
    if y is None and (quant is None if want_y is None else want_y or quant is None):
        y = torch.empty(shape, dtype=x.dtype, device=dev)
    _need(y, "y", dt, shape, optional=True)
    code = 0
    if quant is not None:
        code = _NAME_DT[quant]
        mx = code == _abi.DSA_MXFP8_E4M3
        if mx and d % 32:
            raise ValueError(f"mxfp8 needs a last dimension that is a multiple of 32, not {d}")
        sshape = shape[:-1] + (d // 32,) if mx else shape[:-1]
        if codes is None:
            codes = torch.empty(shape, dtype=torch.uint8, device=dev)
        if scale is None:
            scale = torch.empty(sshape, dtype=torch.uint8 if mx else torch.float32, device=dev)
        _need(codes, "codes", _abi.DSA_FP8_E4M3, shape)
        _need(scale, "scale", _abi.DSA_FP8_E4M3 if mx else _abi.DSA_F32, sshape)
    elif codes is not None or scale is not None:
        raise ValueError("codes and scale need quant")
    _same_device(dev, weight=weight, residual=residual, h=h, y=y, codes=codes, scale=scale)
    with _on(dev):
        _abi.check(lib().dsa_add_rmsnorm(rows, d, dt, code, eps, x.data_ptr(), ld_x,
                                         _ptr(residual), ld_r, weight.data_ptr(), _ptr(h), _ptr(y),
                                         _ptr(codes), _ptr(scale), _stream(dev)))
    return y, h, codes, scale


def prefix_mla_attn(P: Problem, q, kv, prefix_kv=None, prefix_table=None,
                    prefix_len: Optional[int] = None, out=None, lse=None, want_lse: bool = True,
                    ws: Optional[Workspace] = None):
    """Dense MLA attention of all sequences over one shared prefix and, causally, over their own
    latent rows (dsa_prefix_mla_attn): (out[ΣT, H, d_c], lse or None).

    P describes the sequences behind the prefix.  The prefix is prefix_kv [prefix_len, D], or, in a
    paged cache, the pages prefix_table [>= ceil(prefix_len / page_size)] int32 of kv; without
    either there is none."""
    _need(q, "q", P.kv_dtype, (P.total_q, P.h, P.d))
    _need(kv, "kv", P.kv_dtype, (P.cache_rows, P.d))
    dev = kv.device
    if prefix_kv is not None and prefix_table is not None:
        raise ValueError("prefix_kv and prefix_table exclude each other")
    n = 0
    if prefix_kv is not None:
        n = prefix_kv.shape[0] if prefix_len is None else int(prefix_len)
        if prefix_kv.dim() != 2 or not 0 <= n <= prefix_kv.shape[0]:
            raise ValueError(f"prefix_len is {n}, prefix_kv {tuple(prefix_kv.shape)}")
        _need(prefix_kv, "prefix_kv", P.kv_dtype, (prefix_kv.shape[0], P.d))
    elif prefix_table is not None:
        if not P.page_size:
            raise ValueError("prefix_table needs paged caches")
        if prefix_len is None:
            raise ValueError("prefix_table needs prefix_len")
        n = int(prefix_len)
        if not prefix_table.is_cuda or prefix_table.dtype != torch.int32 \
                or prefix_table.dim() != 1 or not prefix_table.is_contiguous() \
                or n < 0 or prefix_table.numel() * P.page_size < n:
            raise ValueError("prefix_table must be a contiguous int32 CUDA tensor that covers prefix_len")
    elif prefix_len:
        raise ValueError("prefix_len needs prefix_kv or prefix_table")
    out, lse = _attn_out(P, out, lse, dev, want_lse)
    _same_device(dev, q=q, prefix_kv=prefix_kv, prefix_table=prefix_table, out=out, lse=lse,
                 cu_q=P.cu_q)
    with _on(dev):
        ws = _op_workspace(ws, dev, P.workspace_size(_abi.OP_PREFIX_MLA_ATTN))
        _abi.check(lib().dsa_prefix_mla_attn(
            ctypes.byref(P.c), n, _ptr(prefix_kv) if n else None, _ptr(prefix_table) if n else None,
            q.data_ptr(), kv.data_ptr(), out.data_ptr(), _ptr(lse), ws.ptr, ws.nbytes,
            _stream(dev)))
    return out, lse


def accumulate_attn_weights(P: Problem, q, kv, idx, lse, acc, ws: Optional[Workspace] = None):
    """Add the attention weight every selected position received, summed over heads and queries,
    to acc [B, >= max_k_len] f32 in place (dsa_accumulate_attn_weights); returns acc.  idx and lse
    are those of sparse_mla_attn or fused_forward on the same q and kv."""
    _need(q, "q", P.kv_dtype, (P.total_q, P.h, P.d))
    _need(kv, "kv", P.kv_dtype, (P.cache_rows, P.d))
    _need(idx, "idx", None, (P.total_q, P.top_k))
    if idx.dtype != torch.int32:
        raise ValueError(f"idx has dtype {idx.dtype}")
    _need(lse, "lse", _abi.DSA_F32, (P.total_q, P.h))
    ld = _acc_stride(P, acc, "acc", P.max_k_len)
    dev = kv.device
    _same_device(dev, q=q, idx=idx, lse=lse, acc=acc, cu_q=P.cu_q)
    with _on(dev):
        ws = _op_workspace(ws, dev, P.workspace_size(_abi.OP_ATTN_WEIGHTS))
        _abi.check(lib().dsa_accumulate_attn_weights(
            ctypes.byref(P.c), q.data_ptr(), kv.data_ptr(), idx.data_ptr(), lse.data_ptr(),
            acc.data_ptr(), ld, ws.ptr, ws.nbytes, _stream(dev)))
    return acc


def _acc_stride(P: Problem, acc, name: str, width: int) -> int:
    """Row stride of an accumulator [B, >= width] f32 (rows contiguous, any stride between)."""
    if not acc.is_cuda or acc.dtype != torch.float32 or acc.dim() != 2 \
            or acc.shape[0] != P.c.num_seqs or acc.shape[1] < width \
            or (acc.shape[1] > 1 and acc.stride(1) != 1) \
            or (acc.shape[0] > 1 and acc.stride(0) < acc.shape[1]):
        raise ValueError(f"{name} must be a float32 CUDA tensor [{P.c.num_seqs}, >= {width}] with "
                         "contiguous rows")
    return acc.stride(0) if acc.shape[0] > 1 else acc.shape[1]


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
    acc_out [B, >= budget] receives the kept positions' acc and zeros behind them."""
    budget, sink, recent = int(budget), int(sink), int(recent)
    if budget < 1 or sink < 0 or recent < 0 or sink + recent > budget:
        raise ValueError(f"budget = {budget}, sink = {sink}, recent = {recent}: 1 <= budget and "
                         "sink + recent <= budget are needed")
    B, dev = P.c.num_seqs, acc.device
    ld = _acc_stride(P, acc, "acc", P.max_k_len)
    k_lens = [min(n, budget) for n in P.k_lens]
    rows = sum(k_lens)
    max_pages = num_pages = 0
    if block_table_out is not None:
        if not P.page_size:
            raise ValueError("block_table_out needs paged caches")
        if not block_table_out.is_cuda or block_table_out.dtype != torch.int32 \
                or block_table_out.dim() != 2 or block_table_out.shape[0] != B \
                or not block_table_out.is_contiguous() \
                or block_table_out.shape[1] * P.page_size < max(k_lens):
            raise ValueError("block_table_out must be a contiguous int32 CUDA tensor [B, pages] that covers "
                             "the kept positions")
        max_pages = block_table_out.shape[1]
    mx = P.idx_dtype == _abi.DSA_MXFP8_E4M3
    codes = _abi.DSA_FP8_E4M3 if mx else P.idx_dtype
    if k_scale is not None and not mx and P.idx_dtype != _abi.DSA_FP8_E4M3:
        raise ValueError("k_scale goes with FP8 or MXFP8 index keys")
    moved = {}
    rows_out = None
    for name, src, dst, code, tail in (
            ("kv", kv, kv_out, P.kv_dtype, (P.d,)),
            ("k_idx", k_idx, k_idx_out, codes, (P.c.d_idx,)),
            ("k_scale", k_scale, k_scale_out, _abi.DSA_FP8_E4M3 if mx else _abi.DSA_F32,
             (P.c.d_idx // 32,) if mx else ())):
        if src is None:
            if dst is not None:
                raise ValueError(f"{name}_out needs {name}")
            moved[name] = None
            continue
        _need(src, name, code, (P.cache_rows,) + tail)
        if dst is None:
            if block_table_out is not None:
                raise ValueError(f"a paged destination needs {name}_out")
            dst = torch.empty((rows,) + tail, dtype=src.dtype, device=dev)
        n = dst.shape[0]
        _need(dst, name + "_out", code, (n,) + tail)
        if n < rows or (rows_out is not None and n != rows_out) \
                or (block_table_out is not None and n % P.page_size):
            raise ValueError(f"{name}_out has {n} rows: all destinations need the same number, at "
                             f"least {rows}, whole pages where they are paged")
        rows_out = n
        moved[name] = dst
    if block_table_out is not None:
        num_pages = (rows_out if rows_out is not None else P.cache_rows) // P.page_size
    if kept is None:
        kept = torch.empty(B, budget, dtype=torch.int32, device=dev)
    if cu_k_out is None:
        cu_k_out = torch.empty(B + 1, dtype=torch.int32, device=dev)
    if acc_out is None:
        acc_out = torch.empty(B, budget, dtype=torch.float32, device=dev)
    for name, t, shape in (("kept", kept, (B, budget)), ("cu_k_out", cu_k_out, (B + 1,))):
        _need(t, name, None, shape)
        if t.dtype != torch.int32:
            raise ValueError(f"{name} has dtype {t.dtype}")
    ld_out = _acc_stride(P, acc_out, "acc_out", budget)
    _same_device(dev, kv=kv, k_idx=k_idx, k_scale=k_scale, kept=kept, cu_k_out=cu_k_out,
                 acc_out=acc_out, block_table_out=block_table_out, cu_k=P.cu_k,
                 **{k + "_out": v for k, v in moved.items()})
    with _on(dev):
        ws = _op_workspace(ws, dev, P.workspace_size(_abi.OP_EVICT))
        _abi.check(lib().dsa_evict(
            ctypes.byref(P.c), acc.data_ptr(), ld, budget, sink, recent, kept.data_ptr(),
            cu_k_out.data_ptr(), acc_out.data_ptr(), ld_out, _ptr(kv), _ptr(moved["kv"]),
            _ptr(k_idx), _ptr(moved["k_idx"]), _ptr(k_scale), _ptr(moved["k_scale"]),
            _ptr(block_table_out), max_pages, num_pages, rows_out or 0, ws.ptr, ws.nbytes,
            _stream(dev)))
    return Eviction(kept, cu_k_out, k_lens, acc_out, moved["kv"], moved["k_idx"], moved["k_scale"])


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
