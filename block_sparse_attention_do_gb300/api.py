"""ctypes binding over libnsa.so (declared in include/nsa.h).

Argument marshalling only: every step of the computation runs in the
library's CUDA kernels.  torch provides device memory (outputs and the
workspace) and the current CUDA stream.  There is no CPU fallback: if the
library is missing the first call raises.
"""
from __future__ import annotations

import ctypes as C
import math
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libnsa.so")

NSA_OK = 0
STATUS = {0: "NSA_OK", 1: "NSA_ERR_INVALID_ARG", 2: "NSA_ERR_UNSUPPORTED", 3: "NSA_ERR_BAD_INDEX",
          4: "NSA_ERR_DEVICE_TIMEOUT", 5: "NSA_ERR_CUDA", 6: "NSA_ERR_WORKSPACE", 7: "NSA_ERR_CACHE_FULL"}
DTYPE = {torch.float32: 0, torch.bfloat16: 1}
LAYOUT_BHTD, LAYOUT_THD = 0, 1

# every entry point of include/nsa.h
SYMBOLS = (
    "nsa_fwd_workspace_size", "nsa_bwd_workspace_size", "nsa_sel_fwd", "nsa_sel_bwd",
    "nsa_dense_causal_fwd", "nsa_dense_causal_bwd", "nsa_sel_varlen_fwd", "nsa_sel_varlen_bwd",
    "nsa_do_dot", "nsa_inverse_index_offsets_len", "nsa_build_inverse_index", "nsa_get_error",
    "nsa_status_string", "nsa_count_pairs", "nsa_trace_enable", "nsa_trace_reset",
    "nsa_trace_count", "nsa_trace_get", "nsa_build_inverse_index_noalloc",
    "nsa_plan_size", "nsa_plan_build", "nsa_bwd_planned_workspace_size", "nsa_sel_bwd_planned",
    "nsa_swa_fwd", "nsa_swa_bwd", "nsa_sink_fwd", "nsa_sink_bwd", "nsa_debug_stall",
    "nsa_causal_fwd_workspace_size", "nsa_causal_bwd_workspace_size", "nsa_causal_fwd", "nsa_causal_bwd",
    "nsa_select_workspace_size", "nsa_compress_keys_mean", "nsa_block_scores", "nsa_select_topk",
    "nsa_sel_fwd_workspace_size", "nsa_sel_bwd_workspace_size",
    "nsa_norm_rope_fwd", "nsa_norm_rope_bwd_workspace_size", "nsa_norm_rope_bwd",
    "nsa_cache_workspace_size", "nsa_cache_reserve", "nsa_cache_free", "nsa_cache_fork", "nsa_cache_copy",
    "nsa_cache_compact", "nsa_cache_append", "nsa_cache_fwd_workspace_size", "nsa_cache_fwd",
    "nsa_cache_tree_fwd_workspace_size", "nsa_cache_tree_fwd", "nsa_cache_accept", "nsa_cache_weigh", "nsa_cache_evict",
)


class Problem(C.Structure):
    _fields_ = [("B", C.c_int32), ("Hq", C.c_int32), ("Hkv", C.c_int32), ("T", C.c_int32),
                ("D", C.c_int32), ("block_size", C.c_int32), ("S", C.c_int32),
                ("dtype", C.c_int32), ("layout", C.c_int32), ("total_tokens", C.c_int32),
                ("scale", C.c_float), ("reserved", C.c_int32),
                ("q_stride", C.c_int64 * 3), ("kv_stride", C.c_int64 * 3), ("o_stride", C.c_int64 * 3),
                ("dq_stride", C.c_int64 * 3), ("dkv_stride", C.c_int64 * 3),
                ("Tk", C.c_int32), ("total_keys", C.c_int32), ("bottom_right", C.c_int32),
                ("reserved2", C.c_int32)]


class CacheStruct(C.Structure):
    """nsa_cache."""
    _fields_ = [("num_pages", C.c_int32), ("Hkv", C.c_int32), ("D", C.c_int32), ("block_size", C.c_int32),
                ("rows", C.c_int32), ("max_pages", C.c_int32), ("stride", C.c_int64 * 3),
                ("k", C.c_void_p), ("v", C.c_void_p), ("k_scale", C.c_void_p), ("v_scale", C.c_void_p),
                ("page_table", C.c_void_p), ("seq_lens", C.c_void_p), ("refcount", C.c_void_p)]


class NormRopeStruct(C.Structure):
    """nsa_norm_rope."""
    _fields_ = [("rotary", C.c_int32), ("interleaved", C.c_int32), ("eps", C.c_float), ("reserved", C.c_int32),
                ("qr_stride", C.c_int64 * 3), ("kr_stride", C.c_int64 * 3)]


def _bht_strides(t, thd):
    """(batch, head, token) element strides of a [B, H, T, D] (or packed
    [total, H, D]) tensor whose last dimension is contiguous."""
    if t.stride(-1) != 1:
        raise ValueError("the head dimension must be contiguous")
    s = (0, t.stride(1), t.stride(0)) if thd else (t.stride(0), t.stride(1), t.stride(2))
    # (all 0 declares a dense tensor: of one row that is expanded, its rows would be read behind it)
    if not any(s) and t.numel() > t.shape[-1]:
        raise ValueError("expanded tensors have no rows of their own: make them contiguous")
    return s


def declare_strides(p: Problem, thd: bool, q=None, k=None, o=None, dq=None, dk=None) -> Problem:
    """Fills the problem's declared strides from the tensors given (k stands
    for k and v, o for o and dO, dk for dk and dv)."""
    for name, t in (("q_stride", q), ("kv_stride", k), ("o_stride", o), ("dq_stride", dq),
                    ("dkv_stride", dk)):
        if t is not None:
            getattr(p, name)[:] = _bht_strides(t, thd)
    return p


def _same_strides(a, b, what):
    if a is not None and b is not None and a.stride() != b.stride():
        raise ValueError(f"{what} must have the same strides")


class NsaError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)}")


_lib = None
_P = C.c_void_p


def lib() -> C.CDLL:
    """Load libnsa.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libnsa.so not built ({LIB_PATH}); run __graft_entry__.build()")
        L = C.CDLL(LIB_PATH)
        pp = C.POINTER(Problem)
        L.nsa_fwd_workspace_size.restype = C.c_size_t
        L.nsa_fwd_workspace_size.argtypes = [pp]
        L.nsa_bwd_workspace_size.restype = C.c_size_t
        L.nsa_bwd_workspace_size.argtypes = [pp]
        L.nsa_sel_fwd.argtypes = [pp] + [_P] * 6 + [_P, C.c_size_t, _P]
        L.nsa_sel_bwd.argtypes = [pp] + [_P] * 10 + [_P, C.c_size_t, _P]
        L.nsa_dense_causal_fwd.argtypes = [pp] + [_P] * 5 + [_P, C.c_size_t, _P]
        L.nsa_dense_causal_bwd.argtypes = [pp] + [_P] * 9 + [_P, C.c_size_t, _P]
        L.nsa_sel_varlen_fwd.argtypes = [pp] + [_P] * 7 + [_P, C.c_size_t, _P]
        L.nsa_sel_varlen_bwd.argtypes = [pp] + [_P] * 11 + [_P, C.c_size_t, _P]
        L.nsa_do_dot.argtypes = [pp] + [_P] * 4 + [_P]
        L.nsa_inverse_index_offsets_len.restype = C.c_int64
        L.nsa_inverse_index_offsets_len.argtypes = [pp]
        L.nsa_build_inverse_index.argtypes = [pp] + [_P] * 4 + [_P, C.c_size_t, _P]
        L.nsa_get_error.argtypes = [_P, _P, C.POINTER(C.c_int32)]
        L.nsa_status_string.restype = C.c_char_p
        L.nsa_status_string.argtypes = [C.c_int32]
        L.nsa_count_pairs.argtypes = [pp] + [_P] * 3 + [_P]
        L.nsa_build_inverse_index_noalloc.argtypes = [pp] + [_P] * 5 + [_P]
        L.nsa_plan_size.restype = C.c_size_t
        L.nsa_plan_size.argtypes = [pp]
        L.nsa_plan_build.argtypes = [pp, _P, _P, _P, C.c_size_t, _P]
        L.nsa_bwd_planned_workspace_size.restype = C.c_size_t
        L.nsa_bwd_planned_workspace_size.argtypes = [pp]
        L.nsa_sel_bwd_planned.argtypes = [pp] + [_P] * 12 + [_P, C.c_size_t, _P]
        L.nsa_swa_fwd.argtypes = [pp, C.c_int32] + [_P] * 6 + [_P, C.c_size_t, _P]
        L.nsa_swa_bwd.argtypes = [pp, C.c_int32] + [_P] * 10 + [_P, C.c_size_t, _P]
        L.nsa_sink_fwd.argtypes = [pp, C.c_int32] + [_P] * 7 + [_P, C.c_size_t, _P]
        L.nsa_sink_bwd.argtypes = [pp, C.c_int32] + [_P] * 12 + [_P, C.c_size_t, _P]
        L.nsa_debug_stall.argtypes = [C.c_int32, C.c_int32]
        L.nsa_causal_fwd_workspace_size.restype = C.c_size_t
        L.nsa_causal_fwd_workspace_size.argtypes = [pp]
        L.nsa_causal_bwd_workspace_size.restype = C.c_size_t
        L.nsa_causal_bwd_workspace_size.argtypes = [pp]
        L.nsa_causal_fwd.argtypes = [pp, C.c_int32] + [_P] * 7 + [_P, C.c_size_t, _P]
        L.nsa_causal_bwd.argtypes = [pp, C.c_int32] + [_P] * 11 + [_P, C.c_size_t, _P]
        L.nsa_trace_enable.argtypes = [C.c_int32]
        L.nsa_trace_reset.restype = None
        L.nsa_trace_reset.argtypes = []
        L.nsa_trace_count.restype = C.c_int32
        L.nsa_trace_count.argtypes = []
        L.nsa_trace_get.argtypes = [C.c_int32, C.POINTER(C.c_char_p), C.POINTER(C.c_float)]
        for name in ("nsa_sel_fwd_workspace_size", "nsa_sel_bwd_workspace_size"):
            getattr(L, name).restype = C.c_size_t
            getattr(L, name).argtypes = [pp]
        L.nsa_select_workspace_size.restype = C.c_size_t
        L.nsa_select_workspace_size.argtypes = [pp]
        L.nsa_compress_keys_mean.argtypes = [pp] + [_P] * 3 + [_P]
        L.nsa_block_scores.argtypes = [pp] + [_P] * 4 + [_P, C.c_size_t, _P]
        L.nsa_select_topk.argtypes = [pp] + [_P] * 3 + [_P]
        pn = C.POINTER(NormRopeStruct)
        L.nsa_norm_rope_fwd.argtypes = [pp, pn] + [_P] * 9 + [_P]
        L.nsa_norm_rope_bwd_workspace_size.restype = C.c_size_t
        L.nsa_norm_rope_bwd_workspace_size.argtypes = [pp]
        L.nsa_norm_rope_bwd.argtypes = [pp, pn] + [_P] * 13 + [_P, C.c_size_t, _P]
        pc = C.POINTER(CacheStruct)
        L.nsa_cache_workspace_size.restype = C.c_size_t
        L.nsa_cache_workspace_size.argtypes = [pc]
        L.nsa_cache_reserve.argtypes = [pc, _P] + [_P, C.c_size_t, _P]
        L.nsa_cache_free.argtypes = [pc, _P, C.c_int32] + [_P, C.c_size_t, _P]
        L.nsa_cache_fork.argtypes = [pc, _P, _P, C.c_int32] + [_P, C.c_size_t, _P]
        L.nsa_cache_copy.argtypes = [pc, _P, _P, C.c_int32] + [_P, C.c_size_t, _P]
        L.nsa_cache_compact.argtypes = [pc] + [_P, C.c_size_t, _P]
        L.nsa_cache_append.argtypes = [pp, pc] + [_P] * 3 + [_P, C.c_size_t, _P]
        L.nsa_cache_fwd_workspace_size.restype = C.c_size_t
        L.nsa_cache_fwd_workspace_size.argtypes = [pp, pc, C.c_int32]
        L.nsa_cache_fwd.argtypes = [pp, pc, C.c_int32] + [_P] * 6 + [_P, C.c_size_t, _P]
        L.nsa_cache_tree_fwd_workspace_size.restype = C.c_size_t
        L.nsa_cache_tree_fwd_workspace_size.argtypes = [pp, pc, C.c_int32]
        L.nsa_cache_tree_fwd.argtypes = [pp, pc, C.c_int32] + [_P] * 7 + [_P, C.c_size_t, _P]
        L.nsa_cache_accept.argtypes = [pc, _P, _P, C.c_int32] + [_P, C.c_size_t, _P]
        L.nsa_cache_weigh.argtypes = [pp, pc, C.c_int32, _P, _P, _P, C.c_float, _P] + [_P, C.c_size_t, _P]
        L.nsa_cache_evict.argtypes = [pc, _P, C.c_int32, C.c_int32, C.c_int32, _P] + [_P, C.c_size_t, _P]
        for name in SYMBOLS:
            fn = getattr(L, name)
            if fn.restype is C.c_int:  # default restype: status enums
                fn.restype = C.c_int32
        _lib = L
    return _lib


def _ptr(t):
    return None if t is None else C.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return C.c_void_p(s.cuda_stream)


def _check(status, where):
    if status != NSA_OK:
        raise NsaError(status, where)


def problem(B, Hq, Hkv, T, D, block_size, S, dtype, layout=LAYOUT_BHTD, total_tokens=0,
            scale=None) -> Problem:
    return Problem(B, Hq, Hkv, T, D, block_size, S, DTYPE[dtype], layout, total_tokens,
                   float(scale) if scale else 0.0)


def problem_from(q, k, block_size, S, scale=None, cu_seqlens=None, max_seqlen=None) -> Problem:
    if cu_seqlens is None:
        B, Hq, T, D = q.shape
        return problem(B, Hq, k.shape[1], T, D, block_size, S, q.dtype, scale=scale)
    total, Hq, D = q.shape
    B = cu_seqlens.numel() - 1
    if max_seqlen is None:
        max_seqlen = int((cu_seqlens[1:] - cu_seqlens[:-1]).max().item()) if B > 0 else 1
    return problem(B, Hq, k.shape[1], max(1, max_seqlen), D, block_size, S, q.dtype,
                   layout=LAYOUT_THD, total_tokens=total, scale=scale)


_ws_cache: dict = {}


def workspace(nbytes: int, device, key="default") -> torch.Tensor:
    """A cached device buffer of at least nbytes (256-byte aligned by torch)."""
    ck = (key, str(device))
    buf = _ws_cache.get(ck)
    if buf is None or buf.numel() < nbytes:
        buf = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
        _ws_cache[ck] = buf
    return buf


def fwd_workspace_size(p: Problem) -> int:
    return int(lib().nsa_fwd_workspace_size(C.byref(p)))


def bwd_workspace_size(p: Problem) -> int:
    return int(lib().nsa_bwd_workspace_size(C.byref(p)))


def bwd_planned_workspace_size(p: Problem) -> int:
    return int(lib().nsa_bwd_planned_workspace_size(C.byref(p)))


def _lse_shape(q, cu_seqlens):
    return q.shape[:-1]


def sel_fwd(q, k, v, block_idx, block_size, scale=None, cu_seqlens=None, max_seqlen=None,
            dense=False, ws=None, stream=None, window=None, sinks=None):
    """Selection (or dense causal, or with `window` sliding-window causal)
    forward through the C ABI: returns (o, lse).  `sinks` (fp32, one logit
    per query head, dense entry only) adds attention sinks."""
    dense = dense or window is not None or sinks is not None
    S = 1 if dense else block_idx.shape[-1]
    p = problem_from(q, k, block_size, S, scale, cu_seqlens, max_seqlen)
    o = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    _same_strides(k, v, "k and v")
    declare_strides(p, cu_seqlens is not None, q=q, k=k, o=o)
    lse = torch.empty(_lse_shape(q, cu_seqlens), dtype=torch.float32, device=q.device)
    n = fwd_workspace_size(p)
    if n == 0:
        raise NsaError(1, "nsa_fwd_workspace_size")
    ws = workspace(n, q.device, "fwd") if ws is None else ws
    L = lib()
    st = _stream(stream)
    if sinks is not None:
        s = L.nsa_sink_fwd(C.byref(p), int(window or 0), _ptr(cu_seqlens), _ptr(sinks), _ptr(q), _ptr(k),
                           _ptr(v), _ptr(o), _ptr(lse), _ptr(ws), ws.numel(), st)
    elif window is not None:
        s = L.nsa_swa_fwd(C.byref(p), int(window), _ptr(cu_seqlens), _ptr(q), _ptr(k), _ptr(v), _ptr(o),
                          _ptr(lse), _ptr(ws), ws.numel(), st)
    elif cu_seqlens is not None:
        s = L.nsa_sel_varlen_fwd(C.byref(p), _ptr(cu_seqlens), _ptr(q), _ptr(k), _ptr(v),
                                 _ptr(block_idx), _ptr(o), _ptr(lse), _ptr(ws), ws.numel(), st)
    elif dense:
        s = L.nsa_dense_causal_fwd(C.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse),
                                   _ptr(ws), ws.numel(), st)
    else:
        s = L.nsa_sel_fwd(C.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(block_idx), _ptr(o),
                          _ptr(lse), _ptr(ws), ws.numel(), st)
    _check(s, "nsa fwd")
    return o, lse


def build_plan(q, k, block_idx, block_size, scale=None, cu_seqlens=None, max_seqlen=None,
               stream=None):
    """A reusable backward plan (device uint8 tensor) of block_idx, for
    sel_bwd(..., plan=...); q and k only give the problem's shapes."""
    p = problem_from(q, k, block_size, block_idx.shape[-1], scale, cu_seqlens, max_seqlen)
    L = lib()
    n = int(L.nsa_plan_size(C.byref(p)))
    if n == 0:
        raise NsaError(1, "nsa_plan_size")
    plan = torch.empty(n, dtype=torch.uint8, device=block_idx.device)
    _check(L.nsa_plan_build(C.byref(p), _ptr(cu_seqlens), _ptr(block_idx), _ptr(plan), plan.numel(),
                            _stream(stream)), "nsa_plan_build")
    return plan


def sel_bwd(q, k, v, o, dO, lse, block_idx, block_size, scale=None, cu_seqlens=None,
            max_seqlen=None, dense=False, ws=None, stream=None, out=None, plan=None, window=None,
            sinks=None):
    """Selection (or dense causal, or with `window` sliding-window causal)
    backward through the C ABI: returns (dq, dk, dv), and dsinks as a fourth
    value with `sinks` (dense entry only; o and lse as the sink forward wrote
    them).  With `plan` (from build_plan on the same block_idx) the index
    build is skipped."""
    dense = dense or window is not None or sinks is not None
    S = 1 if dense else block_idx.shape[-1]
    p = problem_from(q, k, block_size, S, scale, cu_seqlens, max_seqlen)
    if out is None:
        dq = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        dk = torch.empty(k.shape, dtype=k.dtype, device=k.device)
        dv = torch.empty(v.shape, dtype=v.dtype, device=v.device)
    else:
        dq, dk, dv = out
    _same_strides(k, v, "k and v")
    _same_strides(o, dO, "o and dO")
    _same_strides(dk, dv, "dk and dv")
    declare_strides(p, cu_seqlens is not None, q=q, k=k, o=o, dq=dq, dk=dk)
    L = lib()
    if plan is not None:
        if dense:
            raise ValueError("a plan serves the selection backward only")
        n = bwd_planned_workspace_size(p)
        if n == 0:
            raise NsaError(1, "nsa_bwd_planned_workspace_size")
        ws = workspace(n, q.device, "bwd_planned") if ws is None else ws
        s = L.nsa_sel_bwd_planned(C.byref(p), _ptr(cu_seqlens), _ptr(q), _ptr(k), _ptr(v), _ptr(o),
                                  _ptr(dO), _ptr(lse), _ptr(block_idx), _ptr(plan), _ptr(dq), _ptr(dk),
                                  _ptr(dv), _ptr(ws), ws.numel(), _stream(stream))
        _check(s, "nsa_sel_bwd_planned")
        return dq, dk, dv
    n = bwd_workspace_size(p)
    if n == 0:
        raise NsaError(1, "nsa_bwd_workspace_size")
    ws = workspace(n, q.device, "bwd") if ws is None else ws
    st = _stream(stream)
    if sinks is not None:
        dsinks = torch.empty_like(sinks)
        s = L.nsa_sink_bwd(C.byref(p), int(window or 0), _ptr(cu_seqlens), _ptr(sinks), _ptr(q), _ptr(k),
                           _ptr(v), _ptr(o), _ptr(dO), _ptr(lse), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dsinks),
                           _ptr(ws), ws.numel(), st)
        _check(s, "nsa_sink_bwd")
        return dq, dk, dv, dsinks
    if window is not None:
        s = L.nsa_swa_bwd(C.byref(p), int(window), _ptr(cu_seqlens), _ptr(q), _ptr(k), _ptr(v), _ptr(o),
                          _ptr(dO), _ptr(lse), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(ws), ws.numel(), st)
    elif cu_seqlens is not None:
        s = L.nsa_sel_varlen_bwd(C.byref(p), _ptr(cu_seqlens), _ptr(q), _ptr(k), _ptr(v), _ptr(o),
                                 _ptr(dO), _ptr(lse), _ptr(block_idx), _ptr(dq), _ptr(dk),
                                 _ptr(dv), _ptr(ws), ws.numel(), st)
    elif dense:
        s = L.nsa_dense_causal_bwd(C.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dO),
                                   _ptr(lse), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(ws), ws.numel(),
                                   st)
    else:
        s = L.nsa_sel_bwd(C.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dO), _ptr(lse),
                          _ptr(block_idx), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(ws), ws.numel(), st)
    _check(s, "nsa bwd")
    return dq, dk, dv


def _causal_problem(q, k, cu_q, cu_k, max_q, max_k, bottom_right, scale):
    if cu_q is None:
        B, Hq, T, D = q.shape
        p = problem(B, Hq, k.shape[1], T, D, 64, 1, q.dtype, scale=scale)
        p.Tk = k.shape[2]
    else:
        B = cu_q.numel() - 1
        if max_q is None:
            max_q = int((cu_q[1:] - cu_q[:-1]).max().item()) if B > 0 else 1
        if max_k is None:
            max_k = int((cu_k[1:] - cu_k[:-1]).max().item()) if B > 0 else 1
        p = problem(B, q.shape[1], k.shape[1], max(1, max_q), q.shape[2], 64, 1, q.dtype, layout=LAYOUT_THD,
                    total_tokens=q.shape[0], scale=scale)
        p.Tk = max(1, max_k)
        p.total_keys = k.shape[0]
    p.bottom_right = int(bool(bottom_right))
    return p


def causal_fwd(q, k, v, block_size=64, window=0, bottom_right=False, cu_seqlens_q=None, cu_seqlens_k=None,
               max_seqlen_q=None, max_seqlen_k=None, scale=None, ws=None, stream=None):
    """Dense causal attention whose keys have their own lengths
    (nsa_causal_fwd): the diagonal aligned top-left (row t sees keys <= t)
    or bottom-right (keys <= t + Lk - Lq), with an optional window.
    Returns (o, lse)."""
    p = _causal_problem(q, k, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, bottom_right, scale)
    p.block_size = block_size
    o = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    _same_strides(k, v, "k and v")
    declare_strides(p, cu_seqlens_q is not None, q=q, k=k, o=o)
    lse = torch.empty(q.shape[:-1], dtype=torch.float32, device=q.device)
    L = lib()
    n = int(L.nsa_causal_fwd_workspace_size(C.byref(p)))
    if n == 0:
        raise NsaError(1, "nsa_causal_fwd_workspace_size")
    ws = workspace(n, q.device, "fwd") if ws is None else ws
    _check(L.nsa_causal_fwd(C.byref(p), int(window), _ptr(cu_seqlens_q), _ptr(cu_seqlens_k), _ptr(q), _ptr(k),
                            _ptr(v), _ptr(o), _ptr(lse), _ptr(ws), ws.numel(), _stream(stream)), "nsa_causal_fwd")
    return o, lse


def causal_bwd(q, k, v, o, dO, lse, block_size=64, window=0, bottom_right=False, cu_seqlens_q=None,
               cu_seqlens_k=None, max_seqlen_q=None, max_seqlen_k=None, scale=None, ws=None, stream=None,
               out=None):
    """Backward of causal_fwd (nsa_causal_bwd): returns (dq, dk, dv)."""
    p = _causal_problem(q, k, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, bottom_right, scale)
    p.block_size = block_size
    if out is None:
        dq = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        dk = torch.empty(k.shape, dtype=k.dtype, device=k.device)
        dv = torch.empty(v.shape, dtype=v.dtype, device=v.device)
    else:
        dq, dk, dv = out
    _same_strides(k, v, "k and v")
    _same_strides(o, dO, "o and dO")
    _same_strides(dk, dv, "dk and dv")
    declare_strides(p, cu_seqlens_q is not None, q=q, k=k, o=o, dq=dq, dk=dk)
    L = lib()
    n = int(L.nsa_causal_bwd_workspace_size(C.byref(p)))
    if n == 0:
        raise NsaError(1, "nsa_causal_bwd_workspace_size")
    ws = workspace(n, q.device, "bwd") if ws is None else ws
    _check(L.nsa_causal_bwd(C.byref(p), int(window), _ptr(cu_seqlens_q), _ptr(cu_seqlens_k), _ptr(q), _ptr(k),
                            _ptr(v), _ptr(o), _ptr(dO), _ptr(lse), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(ws),
                            ws.numel(), _stream(stream)), "nsa_causal_bwd")
    return dq, dk, dv


def do_dot(o, dO, cu_seqlens=None, stream=None):
    p = problem_from(o, o, 16, 1, None, cu_seqlens)
    _same_strides(o, dO, "o and dO")
    declare_strides(p, cu_seqlens is not None, o=o)
    delta = torch.empty(o.shape[:-1], dtype=torch.float32, device=o.device)
    _check(lib().nsa_do_dot(C.byref(p), _ptr(cu_seqlens), _ptr(o), _ptr(dO), _ptr(delta),
                            _stream(stream)), "nsa_do_dot")
    return delta


def build_inverse_index(block_idx, Hq, block_size, cu_seqlens=None, max_seqlen=None,
                        stream=None):
    """Returns (offsets, rows) device int32 tensors (rows trimmed on the host)."""
    if cu_seqlens is None:
        B, Hkv, T, S = block_idx.shape
        p = problem(B, Hq, Hkv, T, 64, block_size, S, torch.bfloat16)
        ntok = B * T
    else:
        total, Hkv, S = block_idx.shape
        B = cu_seqlens.numel() - 1
        if max_seqlen is None:
            max_seqlen = int((cu_seqlens[1:] - cu_seqlens[:-1]).max().item())
        p = problem(B, Hq, Hkv, max(1, max_seqlen), 64, block_size, S, torch.bfloat16,
                    layout=LAYOUT_THD, total_tokens=total)
        ntok = total
    L = lib()
    noff = int(L.nsa_inverse_index_offsets_len(C.byref(p)))
    offsets = torch.empty(noff, dtype=torch.int32, device=block_idx.device)
    rows = torch.empty(max(1, ntok * Hkv * S), dtype=torch.int32, device=block_idx.device)
    ws = workspace(bwd_workspace_size(p), block_idx.device, "csr")
    _check(L.nsa_build_inverse_index(C.byref(p), _ptr(cu_seqlens), _ptr(block_idx), _ptr(offsets),
                                     _ptr(rows), _ptr(ws), ws.numel(), _stream(stream)),
           "nsa_build_inverse_index")
    return offsets, rows, ws


def get_error(ws, stream=None) -> int:
    out = C.c_int32(0)
    _check(lib().nsa_get_error(_ptr(ws), _stream(stream), C.byref(out)), "nsa_get_error")
    return int(out.value)


def count_pairs(block_idx, Hq, block_size, cu_seqlens=None, max_seqlen=None, stream=None) -> int:
    if cu_seqlens is None:
        B, Hkv, T, S = block_idx.shape
        p = problem(B, Hq, Hkv, T, 64, block_size, S, torch.bfloat16)
    else:
        total, Hkv, S = block_idx.shape
        B = cu_seqlens.numel() - 1
        if max_seqlen is None:
            max_seqlen = int((cu_seqlens[1:] - cu_seqlens[:-1]).max().item())
        p = problem(B, Hq, Hkv, max(1, max_seqlen), 64, block_size, S, torch.bfloat16,
                    layout=LAYOUT_THD, total_tokens=total)
    out = torch.zeros(1, dtype=torch.int64, device=block_idx.device)
    _check(lib().nsa_count_pairs(C.byref(p), _ptr(cu_seqlens), _ptr(block_idx), _ptr(out),
                                 _stream(stream)), "nsa_count_pairs")
    return int(out.item())


def debug_stall(kernel: int, wait_limit_us: int):
    """Self-test of the kernels' bounded waits (nsa_debug_stall): kernel 1
    (forward), 2 (dK/dV) or 3 (dQ) runs with its S-product issuer idle and
    every wait gives up after wait_limit_us; (0, 0) restores normal operation."""
    _check(lib().nsa_debug_stall(int(kernel), int(wait_limit_us)), "nsa_debug_stall")


def trace_enable(max_records: int):
    _check(lib().nsa_trace_enable(int(max_records)), "nsa_trace_enable")


def trace_reset():
    lib().nsa_trace_reset()


def trace_records():
    """[(kernel name, ms)] of the launches recorded since the last reset."""
    L = lib()
    out = []
    name = C.c_char_p()
    ms = C.c_float()
    for i in range(int(L.nsa_trace_count())):
        _check(L.nsa_trace_get(i, C.byref(name), C.byref(ms)), "nsa_trace_get")
        out.append((name.value.decode(), float(ms.value)))
    return out


def default_scale(D):
    return 1.0 / math.sqrt(D)


# ---------------------------------------------------------------- block selection
# The step that produces the index (include/nsa.h states the reading): block
# scores from compressed keys, then the own block and the S - 1 best complete
# blocks per index row.


def _nb(T, block_size):
    return (T + block_size - 1) // block_size


def compress_keys_mean(k, block_size, cu_seqlens=None, max_seqlen=None, stream=None):
    """kc [B, Hkv, nb, D] (k's dtype): the mean of each complete block's keys."""
    p = problem_from(k, k, block_size, 1, None, cu_seqlens, max_seqlen)
    declare_strides(p, cu_seqlens is not None, k=k)
    B = p.B
    kc = torch.empty(B, p.Hkv, _nb(p.T, block_size), p.D, dtype=k.dtype, device=k.device)
    _check(lib().nsa_compress_keys_mean(C.byref(p), _ptr(cu_seqlens), _ptr(k), _ptr(kc), _stream(stream)),
           "nsa_compress_keys_mean")
    return kc


def block_scores(q, kc, block_size, scale=None, cu_seqlens=None, max_seqlen=None, ws=None, stream=None):
    """float32 block scores, [B, Hkv, T, nb] (THD [total, Hkv, nb])."""
    p = problem_from(q, kc, block_size, 1, scale, cu_seqlens, max_seqlen)
    declare_strides(p, cu_seqlens is not None, q=q)
    nb = _nb(p.T, block_size)
    if kc.shape[2] != nb or not kc.is_contiguous():
        raise NsaError(1, "block_scores: kc must be a dense [B, Hkv, ceil(T / block_size), D] tensor")
    shape = (p.B, p.Hkv, p.T, nb) if cu_seqlens is None else (q.shape[0], p.Hkv, nb)
    scores = torch.empty(shape, dtype=torch.float32, device=q.device)
    n = int(lib().nsa_select_workspace_size(C.byref(p)))
    if n == 0:
        raise NsaError(1, "nsa_select_workspace_size")
    ws = workspace(n, q.device, "select") if ws is None else ws
    _check(lib().nsa_block_scores(C.byref(p), _ptr(cu_seqlens), _ptr(q), _ptr(kc), _ptr(scores), _ptr(ws),
                                  ws.numel(), _stream(stream)), "nsa_block_scores")
    return scores


def select_topk(scores, block_size, S, cu_seqlens=None, max_seqlen=None, stream=None):
    """int32 index rows from block scores: [B, Hkv, T, S] (THD [total, Hkv, S])."""
    if cu_seqlens is None:
        B, Hkv, T, nb = scores.shape
        p = problem(B, Hkv, Hkv, T, 32, block_size, S, torch.float32)
        shape = (B, Hkv, T, S)
    else:
        total, Hkv, nb = scores.shape
        B = cu_seqlens.numel() - 1
        if max_seqlen is None:
            max_seqlen = int((cu_seqlens[1:] - cu_seqlens[:-1]).max().item()) if B > 0 else 1
        p = problem(B, Hkv, Hkv, max(1, max_seqlen), 32, block_size, S, torch.float32, layout=LAYOUT_THD,
                    total_tokens=total)
        shape = (total, Hkv, S)
    if nb != _nb(p.T, block_size) or not scores.is_contiguous():
        raise NsaError(1, "select_topk: scores must be dense with ceil(T / block_size) entries per row")
    idx = torch.empty(shape, dtype=torch.int32, device=scores.device)
    _check(lib().nsa_select_topk(C.byref(p), _ptr(cu_seqlens), _ptr(scores), _ptr(idx), _stream(stream)),
           "nsa_select_topk")
    return idx


# ---------------------------------------------------------------- norms and rotation
# What a model does to q and k in front of the calls above (include/nsa.h
# states the formulas): RMS norm of every head, rotation by position.


def _off_device(t, stream):
    """Whether a call has to leave the current device or stream for t's
    device and the caller's stream."""
    return stream is not None or t.get_device() != torch._C._cuda_getDevice()


def _row_strides(t, thd):
    """(batch, head, token) strides of a tensor of heads; those of dimensions
    of size 1 (never stepped) replaced by valid ones."""
    _need(t.stride(-1) == 1, "norm_rope: the head dimension must be contiguous")
    s = [(t.stride(i) if t.shape[i] > 1 else t.shape[-1]) for i in range(t.dim() - 1)]
    _need(any(s), "norm_rope: expanded tensors have no rows of their own (all strides 0 declare a dense one): make them contiguous")
    return (t.shape[-1], s[1], s[0]) if thd else tuple(s)


_ropes: dict = {}  # calls' problems, by shapes and strides alone


def _rope_plan(q, k, x, y, dq, dk, inv_freq, eps, interleaved, cu_seqlens):
    """(nsa_problem, nsa_norm_rope, dense output shapes) of a call: q and k;
    x, y the rotated ones or their gradients; dq, dk (None: forward)."""
    thd = cu_seqlens is not None
    _need(q.dim() == k.dim() == (3 if thd else 4) and q.dtype == k.dtype and q.dtype in DTYPE and q.device.type == "cuda",
          "norm_rope: q [B, Hq, T, D] and k [B, Hkv, T, D] (packed [total, heads, D] with cu_seqlens), alike, on a CUDA device")
    _need(q.shape[-1] == k.shape[-1] and q.shape[0] == k.shape[0] and (thd or q.shape[2] == k.shape[2]),
          "norm_rope: q and k have the same tokens and head dimension")
    _need(inv_freq is None or inv_freq.dim() == 1, "norm_rope: inv_freq [rotary / 2]")
    D, rotary = q.shape[-1], 0 if inv_freq is None else 2 * inv_freq.shape[0]
    if thd:
        _need(cu_seqlens.dim() == 1 and cu_seqlens.numel() >= 2, "norm_rope: cu_seqlens [B + 1]")
        p = problem(cu_seqlens.numel() - 1, q.shape[1], k.shape[1], 1, D, 64, 1, q.dtype, layout=LAYOUT_THD, total_tokens=q.shape[0])
    else:
        p = problem(q.shape[0], q.shape[1], k.shape[1], q.shape[2], D, 64, 1, q.dtype)
    n = NormRopeStruct(rotary, int(bool(interleaved)), float(eps), 0)
    p.q_stride[:], p.kv_stride[:] = _row_strides(q, thd), _row_strides(k, thd)
    for t, like in ((x, q), (y, k), (dq, q), (dk, k)):
        _need(t is None or (t.shape == like.shape and t.dtype == like.dtype), "norm_rope: outputs and gradients are like q and k")
    for into, t in ((n.qr_stride, x), (n.kr_stride, y), (p.dq_stride, dq), (p.dkv_stride, dk)):
        if t is not None:
            into[:] = _row_strides(t, thd)
    ws = int(lib().nsa_norm_rope_bwd_workspace_size(C.byref(p)))
    pos = (q.shape[0],) if thd else (q.shape[0], q.shape[2])
    return p, n, C.byref(p), C.byref(n), torch.Size((D,)), torch.Size((rotary // 2,)), torch.Size(pos), ws


def _norm_rope(q, k, x, y, dq, dk, dense, q_weight, k_weight, inv_freq, pos, eps, interleaved, cu_seqlens):
    """The plan of a call (remembered by shapes and strides; dense: x and y,
    or dq and dk, are this call's own, like q and k and dense) and the
    addresses of its parameters; every tensor's type and device checked."""
    key = (q.shape, q.stride(), k.shape, k.stride(), q.dtype, k.dtype, None if dense and dq is None else (x.shape, x.stride(), y.shape, y.stride(), x.dtype, y.dtype),
           None if dense else (dq.shape, dq.stride(), dk.shape, dk.stride(), dq.dtype, dk.dtype) if dq is not None else dense, dq is None,
           None if inv_freq is None else inv_freq.shape, eps, interleaved, None if cu_seqlens is None else cu_seqlens.shape, q.device)
    plan = _ropes.get(key)
    if plan is None:
        if len(_ropes) >= 256:
            _ropes.clear()
        plan = _ropes[key] = _rope_plan(q, k, x, y, dq, dk, inv_freq, eps, interleaved, cu_seqlens)
    dev, f32, at = q.device, torch.float32, []
    _need(k.device == dev and x.device == dev and y.device == dev and (dq is None or (dq.device == dev and dk.device == dev)), "norm_rope: one device")
    for t, shape in ((q_weight, plan[4]), (k_weight, plan[4]), (inv_freq, plan[5])):
        if t is None:
            at.append(None)
        else:
            _need(t.dtype is f32 and t.shape == shape and t.device == dev and t.is_contiguous(),
                  "norm_rope: weights are float32 [D], inv_freq float32 [rotary / 2], dense, on q's device")
            at.append(t.data_ptr())
    for t, shape in ((pos, plan[6]), (cu_seqlens, None)):
        at.append(None if t is None else _int32(t, "norm_rope: pos, cu_seqlens", dev, shape).data_ptr())
    return plan, at


def _dense_like(t):
    return torch.empty_like(t, memory_format=torch.contiguous_format)  # (a third of torch.empty's time)


def norm_rope_fwd(q, k, q_weight, k_weight, inv_freq, pos=None, eps=1e-6, interleaved=False, cu_seqlens=None, out=None,
                  stream=None):
    """RMS norm of every head of q and k (weights float32 [D], or None: ones)
    and the rotation of their first 2 * len(inv_freq) dimensions (a multiple
    of 16; None: none) by pos * inv_freq: pos int32 [B, T] (packed [total]),
    None: each token's place in its sequence.  Pairs are a half apart, or
    with `interleaved` neighbours.  Returns (q, k) rotated, dense or in `out`
    (which may be (q, k))."""
    if _off_device(q, stream):
        with _there(q, stream):
            return norm_rope_fwd(q, k, q_weight, k_weight, inv_freq, pos, eps, interleaved, cu_seqlens, out)
    qr, kr = out or (_dense_like(q), _dense_like(k))
    if q.numel() == 0:
        return qr, kr
    plan, (qw, kw, f, at, cu) = _norm_rope(q, k, qr, kr, None, None, out is None, q_weight, k_weight, inv_freq, pos, eps, interleaved, cu_seqlens)
    _check(lib().nsa_norm_rope_fwd(plan[2], plan[3], cu, q.data_ptr(), k.data_ptr(), qw, kw, f, at, qr.data_ptr(), kr.data_ptr(),
                                   torch._C._cuda_getCurrentRawStream(q.get_device())), "nsa_norm_rope_fwd")
    return qr, kr


def norm_rope_bwd(q, k, dqr, dkr, q_weight, k_weight, inv_freq, pos=None, eps=1e-6, interleaved=False, cu_seqlens=None,
                  ws=None, out=None, stream=None):
    """Backward of norm_rope_fwd, from its q and k and the gradients of its
    results: returns (dq, dk, dq_weight, dk_weight); a weight that is None
    has None.  dq and dk are dense or `out` (which may be (dqr, dkr)).  A ws
    of the caller's has nsa_norm_rope_bwd_workspace_size bytes."""
    if _off_device(q, stream):
        with _there(q, stream):
            return norm_rope_bwd(q, k, dqr, dkr, q_weight, k_weight, inv_freq, pos, eps, interleaved, cu_seqlens, ws, out)
    dq, dk = out or (_dense_like(q), _dense_like(k))
    if q.numel() == 0:
        return dq, dk, *(None if w is None else torch.zeros_like(w) for w in (q_weight, k_weight))
    plan, (qw, kw, f, at, cu) = _norm_rope(q, k, dqr, dkr, dq, dk, out is None, q_weight, k_weight, inv_freq, pos, eps, interleaved, cu_seqlens)
    dqw = None if q_weight is None else torch.empty_like(q_weight)
    dkw = None if k_weight is None else torch.empty_like(k_weight)
    if ws is None:
        ws = q.new_empty(plan[7], dtype=torch.uint8)
    _need(ws.device == q.device, "norm_rope_bwd: ws is on q's device")
    _check(lib().nsa_norm_rope_bwd(plan[2], plan[3], cu, q.data_ptr(), k.data_ptr(), dqr.data_ptr(), dkr.data_ptr(), qw, kw, f, at,
                                   dq.data_ptr(), dk.data_ptr(), None if dqw is None else dqw.data_ptr(), None if dkw is None else dkw.data_ptr(),
                                   ws.data_ptr(), ws.numel(), torch._C._cuda_getCurrentRawStream(q.get_device())), "nsa_norm_rope_bwd")
    return dq, dk, dqw, dkw


# ---------------------------------------------------------------- paged 8-bit cache
# Serving (include/nsa.h states the layout and every rule): a cache of pages
# in e4m3, one scale per page and kv head.  A step of a served batch is
# cache_reserve (pages for the new tokens), cache_append (their keys and
# values) and cache_fwd (their attention).


def _need(ok, what):
    if not ok:
        raise NsaError(1, what)


def _int32(t, what, device, shape=None):
    _need(t.dtype == torch.int32 and t.is_contiguous() and t.device == device and
          (shape is None or tuple(t.shape) == tuple(shape)), f"{what}: a dense int32 tensor on the call's device is wanted")
    return t


class KVCache:
    """The tensors of one paged 8-bit cache (nsa_cache), all on one device:
    k, v float8_e4m3fn [num_pages, Hkv, block_size, D] (strided, D
    contiguous), k_scale, v_scale float32 [num_pages, Hkv], page_table int32
    [rows, max_pages], seq_lens int32 [rows], refcount int32 [num_pages]
    (None: the caller manages pages itself; no reserve, free, fork or
    compact).  The cache keeps their addresses: they are written in place,
    never replaced.  `ws` is the workspace of the calls that change the cache;
    get_error(cache.ws) reads what the last of them found.  `fwd_ws` is the
    last cache_fwd's workspace (None: it had none), `weigh_ws` the last
    cache_weigh's, for get_error too."""

    def __init__(self, k, v, k_scale, v_scale, page_table, seq_lens, refcount=None):
        _need(k.dim() == 4 and k.shape == v.shape and k.dtype == v.dtype == torch.float8_e4m3fn,
              "KVCache: k and v are float8_e4m3fn [num_pages, Hkv, block_size, D]")
        _need(k.stride(3) == 1 and k.stride() == v.stride() and any(k.stride()[:3]),
              "KVCache: k and v have the same strides, D contiguous, and are not expanded")
        dev = k.device
        for s in (k_scale, v_scale):
            _need(s.dtype == torch.float32 and s.is_contiguous() and tuple(s.shape) == tuple(k.shape[:2]) and s.device == dev,
                  "KVCache: scales are dense float32 [num_pages, Hkv]")
        _need(v.device == dev and page_table.dim() == 2, "KVCache: one device, page_table [rows, max_pages]")
        _int32(page_table, "KVCache: page_table", dev)
        _int32(seq_lens, "KVCache: seq_lens", dev, (page_table.shape[0],))
        if refcount is not None:
            _int32(refcount, "KVCache: refcount", dev, (k.shape[0],))
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.page_table, self.seq_lens, self.refcount = page_table, seq_lens, refcount
        self.device, self.index = dev, dev.index
        s = CacheStruct(k.shape[0], k.shape[1], k.shape[3], k.shape[2], page_table.shape[0], page_table.shape[1])
        if not k.is_contiguous():
            s.stride[:] = k.stride()[:3]
        s.k, s.v, s.k_scale, s.v_scale = k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr()
        s.page_table, s.seq_lens = page_table.data_ptr(), seq_lens.data_ptr()
        s.refcount = refcount.data_ptr() if refcount is not None else None
        self.struct, self.ref = s, C.byref(s)
        n = int(lib().nsa_cache_workspace_size(self.ref))
        if n == 0:
            raise NsaError(1, "nsa_cache_workspace_size")
        self.ws = torch.zeros(n, dtype=torch.uint8, device=dev)
        self.fwd_ws = self.weigh_ws = None
        self._problems = {}

    def problem(self, x, S, scale, cu_seqlens, max_seqlen, selection, query, tree=False):
        """The nsa_problem of a call on x (queries, or new keys), and the
        attention's workspace size; remembered by shape."""
        key = (x.shape, x.stride(), x.dtype, S, scale, max_seqlen, cu_seqlens is None, selection, query, tree)
        got = self._problems.get(key)
        if got is None:
            s = self.struct
            _need(x.dtype in DTYPE and x.shape[-1] == s.D, "cache: float32 or bfloat16 rows of the cache's head dimension")
            _need(x.dim() == (4 if cu_seqlens is None else 3) and (cu_seqlens is not None or x.shape[0] == s.rows),
                  "cache: x is [rows, heads, T, D], or packed [total, heads, D] with cu_seqlens")
            Hq = x.shape[1]
            if cu_seqlens is None:
                p = problem(x.shape[0], Hq, s.Hkv, x.shape[2], s.D, s.block_size, S, x.dtype, scale=scale)
            else:
                p = problem(s.rows, Hq, s.Hkv, max(1, max_seqlen), s.D, s.block_size, S, x.dtype, layout=LAYOUT_THD,
                            total_tokens=x.shape[0], scale=scale)
            n = 0
            if query:
                declare_strides(p, cu_seqlens is not None, q=x)
                size = lib().nsa_cache_tree_fwd_workspace_size if tree else lib().nsa_cache_fwd_workspace_size
                n = int(size(C.byref(p), self.ref, int(selection)))
                if n == 0:
                    raise NsaError(1, "nsa_cache_tree_fwd_workspace_size" if tree else "nsa_cache_fwd_workspace_size")
            else:
                _need(Hq == s.Hkv, "cache: new keys and values have the cache's heads")
                declare_strides(p, cu_seqlens is not None, k=x)
            if len(self._problems) >= 256:
                self._problems.clear()
            got = self._problems[key] = (p, C.byref(p), n, x.shape[:-1], x.is_contiguous())
        return got


def make_cache(num_pages, Hkv, D, block_size, rows, max_pages, device="cuda"):
    """An empty KVCache."""
    dev = torch.device(device)
    shape = (num_pages, Hkv, block_size, D)
    i32 = dict(dtype=torch.int32, device=dev)
    return KVCache(torch.zeros(shape, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn),
                   torch.zeros(shape, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn),
                   torch.ones(num_pages, Hkv, device=dev), torch.ones(num_pages, Hkv, device=dev),
                   torch.full((rows, max_pages), -1, **i32), torch.zeros(rows, **i32), torch.zeros(num_pages, **i32))


def _elsewhere(cache, stream):
    """Whether a call has to leave the current device or stream for the
    cache's device and the caller's stream."""
    return stream is not None or cache.index != torch._C._cuda_getDevice()


def _raw_stream(cache):
    """The current stream of the cache's device (a step of a served batch is
    a few microseconds: the plain handle, without a Stream object)."""
    return torch._C._cuda_getCurrentRawStream(cache.index)


def _there(cache, stream):
    """The caller's stream (else the device's current one) as the context of
    a call, so that what it allocates belongs to that stream."""
    _need(cache.device.type == "cuda" and (stream is None or stream.device == cache.device),
          "cache: a CUDA device's cache, and a stream of that device")
    return torch.cuda.stream(torch.cuda.current_stream(cache.device) if stream is None else stream)


def _cu(cache, cu_seqlens, max_seqlen):
    """The longest of the new tokens' runs, the packed offsets checked."""
    _int32(cu_seqlens, "cache: cu_seqlens", cache.device, (cache.struct.rows + 1,))
    return int((cu_seqlens[1:] - cu_seqlens[:-1]).max().item()) if max_seqlen is None else int(max_seqlen)


def cache_reserve(cache, n_new, stream=None):
    """Row b of the cache grows by n_new[b] tokens (int32 [rows]): pages from
    the pool, lowest ids first, and seq_lens; pages of its own that it holds
    there already (its length was lowered: rejected drafts) are used again.  All rows or, with
    too few free pages (NSA_ERR_CACHE_FULL in cache.ws), none."""
    if _elsewhere(cache, stream):
        with _there(cache, stream):
            return cache_reserve(cache, n_new)
    _int32(n_new, "cache_reserve: n_new", cache.device, (cache.struct.rows,))
    _check(lib().nsa_cache_reserve(cache.ref, n_new.data_ptr(), cache.ws.data_ptr(), cache.ws.numel(), _raw_stream(cache)),
           "nsa_cache_reserve")


def cache_free(cache, rows, stream=None):
    """The listed rows (int32) give back their pages and become empty."""
    if _elsewhere(cache, stream):
        with _there(cache, stream):
            return cache_free(cache, rows)
    _int32(rows, "cache_free: rows", cache.device)
    _check(lib().nsa_cache_free(cache.ref, rows.data_ptr(), rows.numel(), cache.ws.data_ptr(), cache.ws.numel(),
                                _raw_stream(cache)), "nsa_cache_free")


def cache_fork(cache, src, dst, stream=None):
    """Row dst[i] (int32) gives back its pages and continues row src[i]: full
    blocks shared, the last, partly filled one copied."""
    if _elsewhere(cache, stream):
        with _there(cache, stream):
            return cache_fork(cache, src, dst)
    _int32(src, "cache_fork: src", cache.device)
    _int32(dst, "cache_fork: dst", cache.device, src.shape)
    _check(lib().nsa_cache_fork(cache.ref, src.data_ptr(), dst.data_ptr(), src.numel(), cache.ws.data_ptr(),
                                cache.ws.numel(), _raw_stream(cache)), "nsa_cache_fork")


def cache_copy(cache, src, dst, stream=None):
    """Pages src[i] (int32) are copied to pages dst[i], codes and scales."""
    if _elsewhere(cache, stream):
        with _there(cache, stream):
            return cache_copy(cache, src, dst)
    _int32(src, "cache_copy: src", cache.device)
    _int32(dst, "cache_copy: dst", cache.device, src.shape)
    _check(lib().nsa_cache_copy(cache.ref, src.data_ptr(), dst.data_ptr(), src.numel(), cache.ws.data_ptr(),
                                cache.ws.numel(), _raw_stream(cache)), "nsa_cache_copy")


def cache_compact(cache, stream=None):
    """Pages in use move to the front of the pool; table and counts follow."""
    if _elsewhere(cache, stream):
        with _there(cache, stream):
            return cache_compact(cache)
    _check(lib().nsa_cache_compact(cache.ref, cache.ws.data_ptr(), cache.ws.numel(), _raw_stream(cache)), "nsa_cache_compact")


def cache_append(cache, k, v, cu_seqlens=None, max_seqlen=None, stream=None):
    """The new tokens' keys and values ([rows, Hkv, T, D], or packed
    [total, Hkv, D] with cu_seqlens) go, rounded to e4m3, to the last
    positions of their rows; seq_lens counts them already (cache_reserve)."""
    if _elsewhere(cache, stream):
        with _there(cache, stream):
            return cache_append(cache, k, v, cu_seqlens, max_seqlen)
    longest = None if cu_seqlens is None else _cu(cache, cu_seqlens, max_seqlen)
    _need(k.shape == v.shape and k.dtype == v.dtype and k.device == v.device == cache.device,
          "cache_append: k and v alike, on the cache's device")
    _same_strides(k, v, "k and v")
    if k.numel() == 0:
        cache.ws[:4].zero_()  # nothing to do, nothing found
        return
    p = cache.problem(k, 1, None, cu_seqlens, longest, False, False)[1]
    _check(lib().nsa_cache_append(p, cache.ref, cu_seqlens.data_ptr() if cu_seqlens is not None else None, k.data_ptr(),
                                  v.data_ptr(), cache.ws.data_ptr(), cache.ws.numel(), _raw_stream(cache)), "nsa_cache_append")


def cache_fwd(q, cache, block_idx=None, scale=None, cu_seqlens=None, max_seqlen=None, window=None, sinks=None, ws=None,
              stream=None):
    """Attention of the rows' last tokens ([rows, Hq, T, D], or packed
    [total, Hq, D] with cu_seqlens) over the cache: all of it, with `window`
    each token's latest keys, with `block_idx` the selected blocks; `sinks` as
    for sel_fwd.  Returns (o, lse).  A ws of the caller's
    (nsa_cache_fwd_workspace_size) holds the error word that get_error reads;
    without one each call has its own, cache.fwd_ws, except a few short rows'
    (the clustered form): that checks its entries only with a ws of the
    caller's, and else leaves bad ones out unreported."""
    if _elsewhere(cache, stream):
        with _there(cache, stream):
            return cache_fwd(q, cache, block_idx, scale, cu_seqlens, max_seqlen, window, sinks, ws)
    return _cache_fwd(q, cache, None, block_idx, scale, cu_seqlens, max_seqlen, window, sinks, ws)


def _cache_fwd(q, cache, parents, block_idx, scale, cu_seqlens, max_seqlen, window, sinks, ws):
    dev = cache.device
    longest = None if cu_seqlens is None else _cu(cache, cu_seqlens, max_seqlen)
    _need(q.device == dev and (ws is None or ws.device == dev), "cache_fwd: q and ws are on the cache's device")
    _need(q.dim() == (4 if cu_seqlens is None else 3), "cache_fwd: q is [rows, Hq, T, D], or packed [total, Hq, D] with cu_seqlens")
    S = 1
    if block_idx is not None:
        _need(window is None and sinks is None, "cache_fwd: a window or sinks go with the whole cache only")
        S = block_idx.shape[-1]
        head = (q.shape[0], cache.struct.Hkv) + ((q.shape[2],) if cu_seqlens is None else ())
        _int32(block_idx, "cache_fwd: block_idx", dev, head + (S,))
    if sinks is not None:
        _need(sinks.dtype == torch.float32 and sinks.is_contiguous() and tuple(sinks.shape) == (q.shape[1],) and
              sinks.device == dev, "cache_fwd: sinks are float32 [Hq]")
    if parents is not None:
        _int32(parents, "cache_tree_fwd: parents", dev, (q.shape[0],) if cu_seqlens is not None else (q.shape[0], q.shape[2]))
    if q.numel() == 0:
        if ws is None and parents is not None:
            ws = torch.empty(256, dtype=torch.uint8, device=dev)
        cache.fwd_ws = ws
        if ws is not None:
            ws[:4].zero_()
        return torch.empty(q.shape, dtype=q.dtype, device=dev), torch.empty(q.shape[:-1], dtype=torch.float32, device=dev)
    _, p, n, stats, dense = cache.problem(q, S, scale, cu_seqlens, longest, block_idx is not None, True, parents is not None)
    o = torch.empty_like(q) if dense else torch.empty(q.shape, dtype=q.dtype, device=dev)
    lse = torch.empty(stats, dtype=torch.float32, device=dev)
    if ws is None and (n > 256 or parents is not None):  # (a parent that is none would be taken as -1 and nobody hear of it)
        ws = torch.empty(n, dtype=torch.uint8, device=dev)
    cache.fwd_ws = ws
    at, size = (None, 0) if ws is None else (ws.data_ptr(), ws.numel())
    if parents is not None:
        _check(lib().nsa_cache_tree_fwd(p, cache.ref, int(window or 0), None if cu_seqlens is None else cu_seqlens.data_ptr(),
                                        parents.data_ptr(), None if block_idx is None else block_idx.data_ptr(),
                                        None if sinks is None else sinks.data_ptr(), q.data_ptr(), o.data_ptr(), lse.data_ptr(), at,
                                        size, _raw_stream(cache)), "nsa_cache_tree_fwd")
        return o, lse
    _check(lib().nsa_cache_fwd(p, cache.ref, int(window or 0), None if cu_seqlens is None else cu_seqlens.data_ptr(),
                               None if block_idx is None else block_idx.data_ptr(), None if sinks is None else sinks.data_ptr(),
                               q.data_ptr(), o.data_ptr(), lse.data_ptr(), at, size, _raw_stream(cache)), "nsa_cache_fwd")
    return o, lse


def cache_tree_fwd(q, cache, parents, block_idx=None, scale=None, cu_seqlens=None, max_seqlen=None, window=None, sinks=None,
                   ws=None, stream=None):
    """cache_fwd for a tree of drafts: parents (int32 [rows, T], or packed
    [total]) names the draft that each of the new tokens continues, -1: what
    was cached before them.  A draft attends that, its ancestors and itself,
    at the position that its depth gives it.  At most 256 drafts a row.
    get_error(cache.fwd_ws) reads what the call found, with or without a ws
    of the caller's."""
    if _elsewhere(cache, stream):
        with _there(cache, stream):
            return cache_tree_fwd(q, cache, parents, block_idx, scale, cu_seqlens, max_seqlen, window, sinks, ws)
    return _cache_fwd(q, cache, parents, block_idx, scale, cu_seqlens, max_seqlen, window, sinks, ws)


def cache_accept(cache, n_new, path, stream=None):
    """Row b's last n_new[b] tokens (int32 [rows]) were drafted; path (int32
    [rows, max_path], ascending, -1 behind the last) names those that stay.
    Their keys and values move to consecutive positions and seq_lens counts
    them; the other drafts are dropped."""
    if _elsewhere(cache, stream):
        with _there(cache, stream):
            return cache_accept(cache, n_new, path)
    _int32(n_new, "cache_accept: n_new", cache.device, (cache.struct.rows,))
    _int32(path, "cache_accept: path", cache.device)
    _need(path.dim() == 2 and path.shape[0] == cache.struct.rows and path.shape[1] > 0, "cache_accept: path is [rows, max_path]")
    _check(lib().nsa_cache_accept(cache.ref, n_new.data_ptr(), path.data_ptr(), path.shape[1], cache.ws.data_ptr(), cache.ws.numel(),
                                  _raw_stream(cache)), "nsa_cache_accept")


def _weights(cache, weight):
    s = cache.struct
    _need(weight.dtype == torch.float32 and weight.is_contiguous() and weight.device == cache.device and
          tuple(weight.shape) == (s.rows, s.Hkv, s.max_pages), "cache: weight is a dense float32 [rows, Hkv, max_pages] on its device")


def cache_weigh(q, lse, cache, weight, decay=1.0, scale=None, cu_seqlens=None, max_seqlen=None, window=None, ws=None, stream=None):
    """What the queries of a cache_fwd call (q, its lse, scale, window and
    offsets; no block_idx, and no tree's) gave each block of their rows,
    summed over tokens and a kv head's query heads, is added to weight
    (float32 [rows, Hkv, max_pages], in place) times decay.  The error word that get_error reads is
    cache.weigh_ws: ws, the caller's 256 bytes, or the call's own."""
    if _elsewhere(cache, stream):
        with _there(cache, stream):
            return cache_weigh(q, lse, cache, weight, decay, scale, cu_seqlens, max_seqlen, window, ws)
    dev = cache.device
    longest = None if cu_seqlens is None else _cu(cache, cu_seqlens, max_seqlen)
    _need(q.device == dev and (ws is None or ws.device == dev), "cache_weigh: q and ws are on the cache's device")
    _need(q.dim() == (4 if cu_seqlens is None else 3), "cache_weigh: q is [rows, Hq, T, D], or packed [total, Hq, D] with cu_seqlens")
    _need(lse.dtype == torch.float32 and lse.is_contiguous() and lse.device == dev and lse.shape == q.shape[:-1],
          "cache_weigh: lse is a dense float32 of q's rows")
    _weights(cache, weight)
    if ws is None:  # (a page that is none, a wait that gave up: eviction would drop the blocks and nobody hear of it)
        ws = torch.empty(256, dtype=torch.uint8, device=dev)
    cache.weigh_ws = ws
    if q.numel() == 0:
        ws[:4].zero_()
        return
    p = cache.problem(q, 1, scale, cu_seqlens, longest, False, True)[1]
    _check(lib().nsa_cache_weigh(p, cache.ref, int(window or 0), None if cu_seqlens is None else cu_seqlens.data_ptr(), q.data_ptr(),
                                 lse.data_ptr(), float(decay), weight.data_ptr(), ws.data_ptr(), ws.numel(), _raw_stream(cache)),
           "nsa_cache_weigh")


def cache_evict(cache, weight, keep, first=0, recent=1, kept=None, stream=None):
    """Rows of more than `keep` blocks give back all but their first `first`,
    their last `recent` and, of the others, those with the largest weight
    (cache_weigh's, summed over the kv heads); table, weight and lengths close
    up.  kept (int32 [rows, max_pages]), if given, gets the column that each
    column was before."""
    if _elsewhere(cache, stream):
        with _there(cache, stream):
            return cache_evict(cache, weight, keep, first, recent, kept)
    s = cache.struct
    _weights(cache, weight)
    if kept is not None:
        _int32(kept, "cache_evict: kept", cache.device, (s.rows, s.max_pages))
    _check(lib().nsa_cache_evict(cache.ref, weight.data_ptr(), int(keep), int(first), int(recent),
                                 None if kept is None else kept.data_ptr(), cache.ws.data_ptr(), cache.ws.numel(), _raw_stream(cache)),
           "nsa_cache_evict")
