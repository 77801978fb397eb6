"""GB300-native fused attention with an in-kernel relative-position bias (T5 buckets, ALiBi),
padding-free varlen packing, forward and backward.

This module is a thin binding over libfatattn.so (C ABI in include/fat_attn.h), by ctypes and, for the
paged-cache and output-layer calls, a small extension module: it only marshals torch tensors into
pointers and sizes. Every step of the computation runs in the CUDA kernels of the library; there is no
other implementation to fall back to, and a missing or unloadable library raises immediately.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

__all__ = [
    "FatAttnError", "load", "fat_attn_fwd", "fat_attn_fwd_workspace_size", "fat_attn_bwd",
    "fat_attn_bwd_workspace_size",
    "fat_attn_get_device_error", "fat_attn_strerror", "fat_attn_bucket_thresholds",
    "fat_attn_debug_buckets", "fat_attn_debug_set_watchdog", "fat_attn_bwd_stages",
    "fat_attn_bwd_noalloc", "fat_xattn_fwd", "fat_xattn_bwd", "fat_xattn_bwd_workspace_size",
    "fat_xattn_splitkv_num_splits", "fat_rope_apply", "fat_rmsnorm_fwd", "fat_rmsnorm_bwd",
    "fat_cross_entropy", "fat_linear_cross_entropy_fwd", "fat_linear_cross_entropy_bwd",
    "fat_linear_cross_entropy_workspace_size", "fat_paged_plan", "fat_rope_init", "fat_rope_embed",
    "fat_paged_append", "fat_paged_attn", "fat_paged_attn_workspace_size", "fat_paged_tree_plan",
    "fat_paged_tree_attn", "FAT_DEVERR_TIMEOUT_FWD", "FAT_DEVERR_TIMEOUT_BWD", "FAT_DEVERR_INDEX",
    "FAT_DEVERR_SEQLENS", "FAT_DEVERR_PAGES", "LIB_PATH",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libfatattn.so")

FAT_DEVERR_TIMEOUT_FWD = 1
FAT_DEVERR_TIMEOUT_BWD = 2
FAT_DEVERR_SEQLENS = 4
FAT_DEVERR_INDEX = 8
FAT_DEVERR_PAGES = 16


class FatAttnError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        detail = ""
        if code == -4:
            detail = "; " + load().fat_attn_last_error_message().decode()
        super().__init__(f"{where} failed: {code} ({fat_attn_strerror(code)}{detail})")


class _Shape(ctypes.Structure):
    _fields_ = [("total_tokens", ctypes.c_int32), ("num_seqs", ctypes.c_int32),
                ("max_seqlen", ctypes.c_int32), ("num_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("stream", ctypes.c_void_p)]


class _XShape(ctypes.Structure):
    _fields_ = [("total_q", ctypes.c_int32), ("total_k", ctypes.c_int32),
                ("num_seqs", ctypes.c_int32), ("max_seqlen_q", ctypes.c_int32),
                ("max_seqlen_k", ctypes.c_int32), ("num_heads_q", ctypes.c_int32),
                ("num_heads_kv", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("stream", ctypes.c_void_p)]


class _Cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("num_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("num_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("stride_page", ctypes.c_int64),
                ("stride_token", ctypes.c_int64), ("stride_head", ctypes.c_int64)]


class _PlanShape(ctypes.Structure):
    _fields_ = [("num_seqs", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("num_pages", ctypes.c_int32), ("table_width", ctypes.c_int32),
                ("num_free", ctypes.c_int32), ("max_tokens", ctypes.c_int32),
                ("stream", ctypes.c_void_p)]


class _Rope(ctypes.Structure):
    _fields_ = [("rotary_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("amplitude", ctypes.c_float), ("reserved", ctypes.c_int32),
                ("rate", ctypes.c_uint64 * 128)]


class _RopeShape(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int32), ("num_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("x_stride_token", ctypes.c_int64),
                ("x_stride_head", ctypes.c_int64), ("y_stride_token", ctypes.c_int64),
                ("y_stride_head", ctypes.c_int64), ("stream", ctypes.c_void_p)]


class _AppendShape(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int32), ("num_heads_q", ctypes.c_int32),
                ("q_stride_token", ctypes.c_int64), ("q_stride_head", ctypes.c_int64),
                ("k_stride_token", ctypes.c_int64), ("k_stride_head", ctypes.c_int64),
                ("v_stride_token", ctypes.c_int64), ("v_stride_head", ctypes.c_int64),
                ("stream", ctypes.c_void_p)]


class _LinearCeShape(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int32), ("vocab", ctypes.c_int32), ("dim", ctypes.c_int32),
                ("hidden_stride", ctypes.c_int64), ("weight_stride", ctypes.c_int64),
                ("logit_scale", ctypes.c_float), ("z_loss", ctypes.c_float),
                ("stream", ctypes.c_void_p)]


class _TreeShape(ctypes.Structure):
    _fields_ = [("total_q", ctypes.c_int32), ("num_seqs", ctypes.c_int32),
                ("max_seqlen_q", ctypes.c_int32), ("mask_words", ctypes.c_int32),
                ("stream", ctypes.c_void_p)]


class _PagedShape(ctypes.Structure):
    _fields_ = [("total_q", ctypes.c_int32), ("num_seqs", ctypes.c_int32),
                ("max_seqlen_q", ctypes.c_int32), ("max_seqlen_k", ctypes.c_int32),
                ("num_heads_q", ctypes.c_int32), ("table_width", ctypes.c_int32),
                ("stream", ctypes.c_void_p)]


_lib = None


def load(path: Optional[str] = None):
    """Load libfatattn.so (built by __graft_entry__.build()). Raises if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise FileNotFoundError(
            f"{p} not found: build the CUDA library first (python -c 'import __graft_entry__ as g; "
            f"g.build()')")
    lib = ctypes.CDLL(p)
    vp, i32, f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    S = ctypes.POINTER(_Shape)
    lib.fat_attn_fwd.argtypes = [S, vp, vp, vp, vp, i32, i32, i32, vp, vp, i32, f32, vp, vp]
    lib.fat_attn_fwd.restype = i32
    lib.fat_attn_fwd_ws.argtypes = [S, vp, vp, vp, vp, i32, i32, i32, vp, vp, i32, f32, vp, vp,
                                    vp, ctypes.c_size_t]
    lib.fat_attn_fwd_ws.restype = i32
    lib.fat_attn_fwd_workspace_size.argtypes = [S]
    lib.fat_attn_fwd_workspace_size.restype = ctypes.c_size_t
    lib.fat_attn_bwd_workspace_size.argtypes = [S]
    lib.fat_attn_bwd_workspace_size.restype = ctypes.c_size_t
    lib.fat_attn_bwd.argtypes = [S, vp, vp, vp, vp, i32, i32, i32, vp, vp, i32, f32, vp, vp, vp,
                                 vp, ctypes.c_size_t, vp, vp, vp, vp]
    lib.fat_attn_bwd.restype = i32
    lib.fat_attn_bwd_preprocess.argtypes = [S, vp, vp, vp, ctypes.c_size_t, vp, i32]
    lib.fat_attn_bwd_preprocess.restype = i32
    lib.fat_attn_bwd_main.argtypes = [S, vp, vp, vp, vp, i32, i32, i32, vp, vp, i32, f32, vp, vp,
                                      vp, ctypes.c_size_t, vp, vp, vp]
    lib.fat_attn_bwd_main.restype = i32
    lib.fat_attn_bwd_finalize.argtypes = [S, vp, ctypes.c_size_t, f32, vp]
    lib.fat_attn_bwd_finalize.restype = i32
    lib.fat_attn_bwd_noalloc.argtypes = [S, vp, vp, vp, vp, i32, i32, i32, vp, vp, i32, f32, vp,
                                         vp, vp, vp, vp, vp, vp]
    lib.fat_attn_bwd_noalloc.restype = i32
    X = ctypes.POINTER(_XShape)
    lib.fat_xattn_fwd.argtypes = [X, vp, vp, vp, vp, i32, i32, i32, vp, vp, vp, i32, f32, vp, vp]
    lib.fat_xattn_fwd.restype = i32
    lib.fat_xattn_splitkv_num_splits.argtypes = [X]
    lib.fat_xattn_splitkv_num_splits.restype = i32
    lib.fat_xattn_splitkv_workspace_size.argtypes = [X, i32]
    lib.fat_xattn_splitkv_workspace_size.restype = ctypes.c_size_t
    lib.fat_xattn_fwd_splitkv.argtypes = [X, vp, vp, vp, vp, i32, i32, i32, vp, vp, vp, i32, f32,
                                          i32, vp, ctypes.c_size_t, vp, vp]
    lib.fat_xattn_fwd_splitkv.restype = i32
    lib.fat_xattn_bwd_workspace_size.argtypes = [X]
    lib.fat_xattn_bwd_workspace_size.restype = ctypes.c_size_t
    lib.fat_xattn_bwd.argtypes = [X, vp, vp, vp, vp, i32, i32, i32, vp, vp, vp, i32, f32, vp, vp,
                                  vp, vp, ctypes.c_size_t, vp, vp, vp, vp]
    lib.fat_xattn_bwd.restype = i32
    ll = ctypes.c_longlong
    lib.fat_rmsnorm_fwd.argtypes = [ll, i32, vp, vp, f32, vp, vp, vp]
    lib.fat_rmsnorm_fwd.restype = i32
    lib.fat_rmsnorm_bwd.argtypes = [ll, i32, vp, vp, vp, vp, vp, vp, vp]
    lib.fat_rmsnorm_bwd.restype = i32
    lib.fat_cross_entropy.argtypes = [ll, i32, vp, vp, f32, f32, vp, vp, vp, vp]
    lib.fat_cross_entropy.restype = i32
    lib.fat_rope_apply.argtypes = [S, vp, vp, vp, ctypes.c_double, i32]
    lib.fat_rope_apply.restype = i32
    P = ctypes.POINTER
    H = P(_LinearCeShape)
    lib.fat_attn_debug_head_columns.argtypes = [H, i32]
    lib.fat_attn_debug_head_columns.restype = i32
    lib.fat_attn_debug_head_workspace.argtypes = [H, i32, i32, P(ctypes.c_size_t)]
    lib.fat_attn_debug_head_workspace.restype = ctypes.c_size_t
    lib.fat_linear_cross_entropy_workspace_size.argtypes = [H, i32]
    lib.fat_linear_cross_entropy_workspace_size.restype = ctypes.c_size_t
    lib.fat_linear_cross_entropy_fwd.argtypes = [H, vp, vp, vp, vp, ctypes.c_size_t, vp, vp]
    lib.fat_linear_cross_entropy_fwd.restype = i32
    lib.fat_linear_cross_entropy_bwd.argtypes = [H, vp, vp, vp, vp, vp, f32, vp, ctypes.c_size_t, vp,
                                                 vp]
    lib.fat_linear_cross_entropy_bwd.restype = i32
    lib.fat_paged_plan.argtypes = [P(_PlanShape)] + [vp] * 9
    lib.fat_paged_plan.restype = i32
    f64 = ctypes.c_double
    lib.fat_rope_init.argtypes = [P(_Rope), i32, i32, f64, f64, f64, f64, f64, f64]
    lib.fat_rope_init.restype = i32
    lib.fat_rope_embed.argtypes = [P(_RopeShape), P(_Rope), vp, vp, vp, i32]
    lib.fat_rope_embed.restype = i32
    lib.fat_paged_append.argtypes = [P(_AppendShape), P(_Cache), P(_Rope)] + [vp] * 6
    lib.fat_paged_append.restype = i32
    lib.fat_paged_attn.argtypes = [P(_PagedShape), P(_Cache), vp, vp, vp, vp, vp, i32, i32, i32,
                                   vp, i32, f32, vp, ctypes.c_size_t, vp, vp]
    lib.fat_paged_attn.restype = i32
    lib.fat_paged_tree_plan.argtypes = [P(_TreeShape)] + [vp] * 5
    lib.fat_paged_tree_plan.restype = i32
    lib.fat_paged_tree_attn.argtypes = [P(_PagedShape), P(_Cache)] + [vp] * 6 + [
        i32, vp, i32, i32, i32, vp, f32, vp, ctypes.c_size_t, vp, vp]
    lib.fat_paged_tree_attn.restype = i32
    lib.fat_paged_attn_workspace_size.argtypes = [P(_PagedShape), P(_Cache)]
    lib.fat_paged_attn_workspace_size.restype = ctypes.c_size_t
    lib.fat_attn_get_device_error.argtypes = [vp, ctypes.POINTER(i32)]
    lib.fat_attn_get_device_error.restype = i32
    lib.fat_attn_strerror.argtypes = [i32]
    lib.fat_attn_strerror.restype = ctypes.c_char_p
    lib.fat_attn_last_error_message.argtypes = []
    lib.fat_attn_last_error_message.restype = ctypes.c_char_p
    lib.fat_attn_bucket_thresholds.argtypes = [i32, i32, i32, ctypes.POINTER(ctypes.c_int32),
                                               ctypes.POINTER(i32), ctypes.POINTER(i32)]
    lib.fat_attn_bucket_thresholds.restype = i32
    lib.fat_attn_debug_buckets.argtypes = [ctypes.c_longlong, i32, i32, i32, i32, vp, vp]
    lib.fat_attn_debug_buckets.restype = i32
    lib.fat_attn_debug_set_watchdog.argtypes = [ctypes.c_longlong, i32]
    lib.fat_attn_debug_set_watchdog.restype = None
    _lib = lib
    return lib


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream_ptr(stream, device) -> int:
    import torch
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _on(device):
    """Context that makes `device` the current CUDA device for the duration of a library call:
    the library launches on, and looks up its per-GPU state for, the current device."""
    import torch
    return torch.cuda.device(device)


def _shape(total_tokens, num_seqs, max_seqlen, num_heads, head_dim, stream_ptr) -> _Shape:
    return _Shape(int(total_tokens), int(num_seqs), int(max_seqlen), int(num_heads),
                  int(head_dim), stream_ptr)


def _check_tensor(name, t, dtype, ndim=None):
    import torch
    if t is None:
        return
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor")


def fat_attn_fwd(q, k, v, cu_seqlens, max_seqlen: int, bias_table=None, num_buckets: int = 0,
                 max_distance: int = 0, bidirectional: bool = True, alibi_slopes=None,
                 causal: bool = False, softmax_scale: float = 1.0, out=None, lse=None,
                 workspace=None, stream=None):
    """Forward pass. q, k, v: bf16 [T, H, d] (CUDA, contiguous); cu_seqlens: int32 [n+1] (CUDA).
    workspace: device bytes for a split last wave (fat_attn_fwd_workspace_size); None allocates
    what the shape uses, False runs without one. Returns (out bf16 [T, H, d], lse fp32 [H, T])."""
    import torch
    lib = load()
    T, H, d = q.shape
    for name, t in (("q", q), ("k", k), ("v", v), ("out", out)):
        _check_tensor(name, t, torch.bfloat16, 3)
    _check_tensor("cu_seqlens", cu_seqlens, torch.int32, 1)
    _check_tensor("bias_table", bias_table, torch.float32)
    _check_tensor("alibi_slopes", alibi_slopes, torch.float32)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((H, T), dtype=torch.float32, device=q.device)
    sh = _shape(T, cu_seqlens.numel() - 1, max_seqlen, H, d, _stream_ptr(stream, q.device))
    args = (ctypes.byref(sh), _ptr(q), _ptr(k), _ptr(v), _ptr(bias_table), int(num_buckets),
            int(max_distance), int(bool(bidirectional)), _ptr(alibi_slopes), _ptr(cu_seqlens),
            int(bool(causal)), float(softmax_scale), _ptr(out), _ptr(lse))
    if workspace is None and not causal:
        need = int(lib.fat_attn_fwd_workspace_size(ctypes.byref(sh)))
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    with _on(q.device):
        if workspace is None or workspace is False:
            rc = lib.fat_attn_fwd(*args)
        else:
            rc = lib.fat_attn_fwd_ws(*args, _ptr(workspace),
                                     int(workspace.numel() * workspace.element_size()))
    if rc != 0:
        raise FatAttnError(rc, "fat_attn_fwd")
    return out, lse


def fat_attn_fwd_workspace_size(total_tokens: int, num_seqs: int, max_seqlen: int,
                                num_heads: int, head_dim: int) -> int:
    """Device bytes that let the forward split its last wave for this shape (0: none)."""
    sh = _shape(total_tokens, num_seqs, max_seqlen, num_heads, head_dim, None)
    return int(load().fat_attn_fwd_workspace_size(ctypes.byref(sh)))


def fat_attn_bwd_workspace_size(total_tokens: int, num_heads: int, head_dim: int,
                                num_seqs: int = 1, max_seqlen: int = 1) -> int:
    """Backward workspace bytes. With the defaults: the minimum every backward call accepts (dQ
    accumulator and D); with the problem's num_seqs and max_seqlen: the size for its fastest
    schedule (adds the rows of a split last wave when the shape has one)."""
    lib = load()
    sh = _shape(total_tokens, num_seqs, max_seqlen, num_heads, head_dim, None)
    return int(lib.fat_attn_bwd_workspace_size(ctypes.byref(sh)))


def fat_attn_bwd(q, k, v, cu_seqlens, max_seqlen: int, out, lse, dout, bias_table=None,
                 num_buckets: int = 0, max_distance: int = 0, bidirectional: bool = True,
                 alibi_slopes=None, causal: bool = False, softmax_scale: float = 1.0,
                 want_dbias: bool = True, workspace=None, dq=None, dk=None, dv=None,
                 dbias_table=None, stream=None):
    """Backward pass of sum(out * dout). Returns (dq, dk, dv, dbias_table or None)."""
    import torch
    lib = load()
    T, H, d = q.shape
    for name, t in (("q", q), ("k", k), ("v", v), ("out", out), ("dout", dout), ("dq", dq),
                    ("dk", dk), ("dv", dv)):
        _check_tensor(name, t, torch.bfloat16, 3)
    _check_tensor("lse", lse, torch.float32, 2)
    _check_tensor("cu_seqlens", cu_seqlens, torch.int32, 1)
    _check_tensor("bias_table", bias_table, torch.float32)
    _check_tensor("alibi_slopes", alibi_slopes, torch.float32)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    if dbias_table is None and want_dbias and bias_table is not None:
        dbias_table = torch.empty_like(bias_table)
    sh = _shape(T, cu_seqlens.numel() - 1, max_seqlen, H, d, _stream_ptr(stream, q.device))
    need = int(lib.fat_attn_bwd_workspace_size(ctypes.byref(sh)))
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    with _on(q.device):
        rc = lib.fat_attn_bwd(ctypes.byref(sh), _ptr(q), _ptr(k), _ptr(v), _ptr(bias_table),
                              int(num_buckets), int(max_distance), int(bool(bidirectional)),
                              _ptr(alibi_slopes), _ptr(cu_seqlens), int(bool(causal)),
                              float(softmax_scale), _ptr(out), _ptr(lse), _ptr(dout),
                              _ptr(workspace), int(workspace.numel() * workspace.element_size()),
                              _ptr(dq), _ptr(dk), _ptr(dv),
                              _ptr(dbias_table))
    if rc != 0:
        raise FatAttnError(rc, "fat_attn_bwd")
    return dq, dk, dv, dbias_table


def fat_attn_bwd_stages(q, k, v, cu_seqlens, max_seqlen: int, out, lse, dout, workspace, dq, dk,
                        dv, dbias_table=None, bias_table=None, num_buckets: int = 0,
                        max_distance: int = 0, bidirectional: bool = True, alibi_slopes=None,
                        causal: bool = False, softmax_scale: float = 1.0, stream=None,
                        between=None):
    """The backward as its three C-ABI stages (preprocess, main, finalize) with every buffer
    supplied by the caller. `between(i)` (optional) is called after enqueueing stage i, e.g. to
    record CUDA events around the main kernel."""
    lib = load()
    T, H, d = q.shape
    sh = _shape(T, cu_seqlens.numel() - 1, max_seqlen, H, d, _stream_ptr(stream, q.device))
    nbytes = int(workspace.numel() * workspace.element_size())
    if between is not None:
        between(-1)
    with _on(q.device):
        rc = lib.fat_attn_bwd_preprocess(ctypes.byref(sh), _ptr(out), _ptr(dout), _ptr(workspace),
                                         nbytes, _ptr(dbias_table), int(num_buckets))
    if rc != 0:
        raise FatAttnError(rc, "fat_attn_bwd_preprocess")
    if between is not None:
        between(0)
    with _on(q.device):
        rc = lib.fat_attn_bwd_main(ctypes.byref(sh), _ptr(q), _ptr(k), _ptr(v), _ptr(bias_table),
                                   int(num_buckets), int(max_distance), int(bool(bidirectional)),
                                   _ptr(alibi_slopes), _ptr(cu_seqlens), int(bool(causal)),
                                   float(softmax_scale), _ptr(lse), _ptr(dout), _ptr(workspace),
                                   nbytes, _ptr(dk), _ptr(dv), _ptr(dbias_table))
    if rc != 0:
        raise FatAttnError(rc, "fat_attn_bwd_main")
    if between is not None:
        between(1)
    with _on(q.device):
        rc = lib.fat_attn_bwd_finalize(ctypes.byref(sh), _ptr(workspace), nbytes,
                                       float(softmax_scale), _ptr(dq))
    if rc != 0:
        raise FatAttnError(rc, "fat_attn_bwd_finalize")
    if between is not None:
        between(2)
    return dq, dk, dv, dbias_table


def fat_attn_bwd_noalloc(q, k, v, cu_seqlens, max_seqlen: int, out, lse, dout, dq, dk, dv,
                         dbias_table=None, bias_table=None, num_buckets: int = 0,
                         max_distance: int = 0, bidirectional: bool = True, alibi_slopes=None,
                         causal: bool = False, softmax_scale: float = 1.0, stream=None):
    """The backward with the library's built-in scratch instead of a workspace, for callers that
    cannot allocate device memory (see fat_attn_bwd_noalloc in include/fat_attn.h). All output
    buffers are supplied by the caller; nothing is allocated here."""
    lib = load()
    T, H, d = q.shape
    sh = _shape(T, cu_seqlens.numel() - 1, max_seqlen, H, d, _stream_ptr(stream, q.device))
    with _on(q.device):
        rc = lib.fat_attn_bwd_noalloc(ctypes.byref(sh), _ptr(q), _ptr(k), _ptr(v), _ptr(bias_table),
                                      int(num_buckets), int(max_distance), int(bool(bidirectional)),
                                      _ptr(alibi_slopes), _ptr(cu_seqlens), int(bool(causal)),
                                      float(softmax_scale), _ptr(out), _ptr(lse), _ptr(dout),
                                      _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dbias_table))
    if rc != 0:
        raise FatAttnError(rc, "fat_attn_bwd_noalloc")
    return dq, dk, dv, dbias_table


def _xshape(q, k, cu_seqlens_q, max_seqlen_q, max_seqlen_k, stream) -> _XShape:
    Tq, Hq, d = q.shape
    Tk, Hkv, _ = k.shape
    return _XShape(int(Tq), int(Tk), int(cu_seqlens_q.numel() - 1), int(max_seqlen_q),
                   int(max_seqlen_k), int(Hq), int(Hkv), int(d), _stream_ptr(stream, q.device))


def fat_xattn_fwd(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q: int, max_seqlen_k: int,
                  bias_table=None, num_buckets: int = 0, max_distance: int = 0,
                  bidirectional: bool = True, alibi_slopes=None, causal: bool = False,
                  softmax_scale: float = 1.0, out=None, lse=None, num_splits: int = 1,
                  workspace=None, stream=None):
    """Forward with its own query and key lengths per document (cross-attention, decode over a
    key cache) and grouped-query heads. q: bf16 [Tq, Hq, d]; k, v: bf16 [Tk, Hkv, d];
    cu_seqlens_q / cu_seqlens_k: int32 [n + 1]. num_splits > 1 splits every document's keys
    into that many ranges (merged by a second grid); 0 lets the library choose.
    Returns (out bf16 [Tq, Hq, d], lse fp32 [Hq, Tq])."""
    import torch
    lib = load()
    for name, t in (("q", q), ("k", k), ("v", v), ("out", out)):
        _check_tensor(name, t, torch.bfloat16, 3)
    for name, t in (("cu_seqlens_q", cu_seqlens_q), ("cu_seqlens_k", cu_seqlens_k)):
        _check_tensor(name, t, torch.int32, 1)
    _check_tensor("bias_table", bias_table, torch.float32)
    _check_tensor("alibi_slopes", alibi_slopes, torch.float32)
    Tq, Hq, d = q.shape
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((Hq, Tq), dtype=torch.float32, device=q.device)
    sh = _xshape(q, k, cu_seqlens_q, max_seqlen_q, max_seqlen_k, stream)
    args = (_ptr(q), _ptr(k), _ptr(v), _ptr(bias_table), int(num_buckets), int(max_distance),
            int(bool(bidirectional)), _ptr(alibi_slopes), _ptr(cu_seqlens_q), _ptr(cu_seqlens_k),
            int(bool(causal)), float(softmax_scale))
    with _on(q.device):
        if num_splits == 0:
            num_splits = int(lib.fat_xattn_splitkv_num_splits(ctypes.byref(sh)))
        if num_splits == 1:
            rc = lib.fat_xattn_fwd(ctypes.byref(sh), *args, _ptr(out), _ptr(lse))
        else:
            need = int(lib.fat_xattn_splitkv_workspace_size(ctypes.byref(sh), int(num_splits)))
            if workspace is None:
                workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
            rc = lib.fat_xattn_fwd_splitkv(ctypes.byref(sh), *args, int(num_splits),
                                           _ptr(workspace),
                                           int(workspace.numel() * workspace.element_size()),
                                           _ptr(out), _ptr(lse))
    if rc != 0:
        raise FatAttnError(rc, "fat_xattn_fwd")
    return out, lse


def fat_xattn_splitkv_num_splits(q, k, cu_seqlens_q, max_seqlen_q: int, max_seqlen_k: int) -> int:
    """The number of key splits the library suggests for this problem."""
    sh = _xshape(q, k, cu_seqlens_q, max_seqlen_q, max_seqlen_k, None)
    return int(load().fat_xattn_splitkv_num_splits(ctypes.byref(sh)))


def fat_xattn_bwd_workspace_size(total_q: int, total_k: int, num_heads_q: int,
                                 num_heads_kv: int, head_dim: int) -> int:
    sh = _XShape(int(total_q), int(total_k), 1, 1, 1, int(num_heads_q), int(num_heads_kv),
                 int(head_dim), None)
    return int(load().fat_xattn_bwd_workspace_size(ctypes.byref(sh)))


def fat_xattn_bwd(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q: int, max_seqlen_k: int,
                  out, lse, dout, bias_table=None, num_buckets: int = 0, max_distance: int = 0,
                  bidirectional: bool = True, alibi_slopes=None, causal: bool = False,
                  softmax_scale: float = 1.0, want_dbias: bool = True, workspace=None, dq=None,
                  dk=None, dv=None, dbias_table=None, stream=None):
    """Backward of sum(out * dout) for fat_xattn_fwd. Returns (dq, dk, dv, dbias or None)."""
    import torch
    lib = load()
    for name, t in (("q", q), ("k", k), ("v", v), ("out", out), ("dout", dout), ("dq", dq),
                    ("dk", dk), ("dv", dv)):
        _check_tensor(name, t, torch.bfloat16, 3)
    _check_tensor("lse", lse, torch.float32, 2)
    for name, t in (("cu_seqlens_q", cu_seqlens_q), ("cu_seqlens_k", cu_seqlens_k)):
        _check_tensor(name, t, torch.int32, 1)
    _check_tensor("bias_table", bias_table, torch.float32)
    _check_tensor("alibi_slopes", alibi_slopes, torch.float32)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    if dbias_table is None and want_dbias and bias_table is not None:
        dbias_table = torch.empty_like(bias_table)
    sh = _xshape(q, k, cu_seqlens_q, max_seqlen_q, max_seqlen_k, stream)
    need = int(lib.fat_xattn_bwd_workspace_size(ctypes.byref(sh)))
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    with _on(q.device):
        rc = lib.fat_xattn_bwd(ctypes.byref(sh), _ptr(q), _ptr(k), _ptr(v), _ptr(bias_table),
                               int(num_buckets), int(max_distance), int(bool(bidirectional)),
                               _ptr(alibi_slopes), _ptr(cu_seqlens_q), _ptr(cu_seqlens_k),
                               int(bool(causal)), float(softmax_scale), _ptr(out), _ptr(lse),
                               _ptr(dout), _ptr(workspace),
                               int(workspace.numel() * workspace.element_size()), _ptr(dq),
                               _ptr(dk), _ptr(dv), _ptr(dbias_table))
    if rc != 0:
        raise FatAttnError(rc, "fat_xattn_bwd")
    return dq, dk, dv, dbias_table


def fat_rope_apply(x, cu_seqlens, max_seqlen: int, base: float = 10000.0, inverse: bool = False,
                   out=None, stream=None):
    """Rotary position embedding of bf16 [T, H, d] rows, positions local to each document
    (inverse=True turns a gradient back). out may be x itself (in place). Returns out."""
    import torch
    lib = load()
    _check_tensor("x", x, torch.bfloat16, 3)
    _check_tensor("out", out, torch.bfloat16, 3)
    _check_tensor("cu_seqlens", cu_seqlens, torch.int32, 1)
    if out is None:
        out = torch.empty_like(x)
    T, H, d = x.shape
    sh = _shape(T, cu_seqlens.numel() - 1, max_seqlen, H, d, _stream_ptr(stream, x.device))
    with _on(x.device):
        rc = lib.fat_rope_apply(ctypes.byref(sh), _ptr(x), _ptr(out), _ptr(cu_seqlens),
                                float(base), int(bool(inverse)))
    if rc != 0:
        raise FatAttnError(rc, "fat_rope_apply")
    return out


def fat_rmsnorm_fwd(x, weight, eps: float = 1e-6, y=None, rstd=None, stream=None):
    """RMSNorm of the rows of x (bf16 [..., dim], contiguous) with an fp32 weight [dim].
    Returns (y bf16 like x, rstd fp32 [rows])."""
    import torch
    lib = load()
    _check_tensor("x", x, torch.bfloat16)
    _check_tensor("weight", weight, torch.float32, 1)
    dim = x.shape[-1]
    rows = x.numel() // dim if dim else 0
    y = torch.empty_like(x) if y is None else y
    rstd = torch.empty(rows, dtype=torch.float32, device=x.device) if rstd is None else rstd
    with _on(x.device):
        rc = lib.fat_rmsnorm_fwd(rows, int(dim), _ptr(x), _ptr(weight), float(eps), _ptr(y),
                                 _ptr(rstd), _stream_ptr(stream, x.device))
    if rc != 0:
        raise FatAttnError(rc, "fat_rmsnorm_fwd")
    return y, rstd


def fat_rmsnorm_bwd(x, weight, rstd, dy, dx=None, dweight=None, stream=None):
    """Gradients of sum(y * dy) for fat_rmsnorm_fwd: (dx bf16 like x, dweight fp32 [dim])."""
    import torch
    lib = load()
    for name, t in (("x", x), ("dy", dy), ("dx", dx)):
        _check_tensor(name, t, torch.bfloat16)
    _check_tensor("weight", weight, torch.float32, 1)
    _check_tensor("rstd", rstd, torch.float32, 1)
    dim = x.shape[-1]
    rows = x.numel() // dim if dim else 0
    dx = torch.empty_like(x) if dx is None else dx
    dweight = torch.empty_like(weight) if dweight is None else dweight
    with _on(x.device):
        rc = lib.fat_rmsnorm_bwd(rows, int(dim), _ptr(x), _ptr(weight), _ptr(rstd), _ptr(dy),
                                 _ptr(dx), _ptr(dweight), _stream_ptr(stream, x.device))
    if rc != 0:
        raise FatAttnError(rc, "fat_rmsnorm_bwd")
    return dx, dweight


def fat_cross_entropy(logits, target, z_loss: float = 0.0, grad_scale: float = 1.0,
                      want_grad: bool = True, loss=None, lse=None, dlogits=None, stream=None):
    """Cross-entropy with a z-loss term per row of logits (bf16 [rows, vocab]) against int32
    targets [rows] (negative = ignored); with want_grad the gradient of grad_scale * sum(loss)
    comes from the same pass. Returns (loss fp32 [rows], lse fp32 [rows], dlogits or None)."""
    import torch
    lib = load()
    _check_tensor("logits", logits, torch.bfloat16, 2)
    _check_tensor("target", target, torch.int32, 1)
    rows, vocab = logits.shape
    loss = torch.empty(rows, dtype=torch.float32, device=logits.device) if loss is None else loss
    lse = torch.empty(rows, dtype=torch.float32, device=logits.device) if lse is None else lse
    if want_grad and dlogits is None:
        dlogits = torch.empty_like(logits)
    with _on(logits.device):
        rc = lib.fat_cross_entropy(int(rows), int(vocab), _ptr(logits), _ptr(target),
                                   float(z_loss), float(grad_scale), _ptr(loss), _ptr(lse),
                                   _ptr(dlogits) if want_grad else None,
                                   _stream_ptr(stream, logits.device))
    if rc != 0:
        raise FatAttnError(rc, "fat_cross_entropy")
    return loss, lse, (dlogits if want_grad else None)


# ---- paged key/value cache, output layer ---------------------------------------------------------
# These calls serve single decode steps, where the host's time counts: their arguments are checked
# and handed to the library by the extension module of csrc/paged_binding.cpp, in order.

CALLS_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_paged_calls.so")
_calls = None


def _load_calls():
    """The extension module, bound to the loaded library (built by __graft_entry__.build())."""
    global _calls
    if _calls is None:
        import importlib.machinery
        import importlib.util

        import torch  # noqa: F401  (the module is linked against its libraries)
        load()
        if not os.path.exists(CALLS_PATH):
            raise FileNotFoundError(f"{CALLS_PATH} not found: build the library first (python -c "
                                    f"'import __graft_entry__ as g; g.build()')")
        loader = importlib.machinery.ExtensionFileLoader("_paged_calls", CALLS_PATH)
        module = importlib.util.module_from_spec(
            importlib.util.spec_from_loader("_paged_calls", loader))
        loader.exec_module(module)
        module.bind(_lib._name, _Rope)
        _calls = module
    return _calls


def _stream_arg(stream):
    return stream if stream is None else int(getattr(stream, "cuda_stream", stream))


def fat_linear_cross_entropy_workspace_size(rows: int, vocab: int, dim: int,
                                            backward: bool = False) -> int:
    """Workspace bytes of fat_linear_cross_entropy_fwd (or _bwd) on the current device, for calls of up to
    `rows` rows."""
    return (_calls or _load_calls()).lce_workspace(rows, vocab, dim, backward)


def fat_linear_cross_entropy_fwd(hidden, weight, target, z_loss: float = 0.0,
                                 logit_scale: float = 1.0, loss=None, lse=None, workspace=None,
                                 stream=None):
    """Cross-entropy (with a z-loss term) of the logits logit_scale * hidden @ weight.T, which are not
    kept: hidden bf16 [rows, dim] and weight bf16 [vocab, dim] (rows may be strided), target int32
    [rows] (negative: ignored). With few rows minus the loss is the score (log-probability) of drafted
    tokens. workspace: fat_linear_cross_entropy_workspace_size bytes (None: allocated here), for one
    call at a time. Returns (loss fp32 [rows], lse fp32 [rows])."""
    r = (_calls or _load_calls()).lce_fwd(hidden, weight, target, z_loss, logit_scale, loss, lse,
                                          workspace, _stream_arg(stream))
    if type(r) is int:
        raise FatAttnError(r, "fat_linear_cross_entropy_fwd")
    return r


def fat_linear_cross_entropy_bwd(hidden, weight, target, lse, dloss=None, z_loss: float = 0.0,
                                 logit_scale: float = 1.0, grad_scale: float = 1.0,
                                 want_dhidden: bool = True, want_dweight: bool = True, dhidden=None,
                                 dweight=None, workspace=None, stream=None):
    """Gradients of grad_scale * sum(dloss * loss) for fat_linear_cross_entropy_fwd (dloss fp32 [rows];
    None: ones), from its lse; the logits are computed again, a piece of the vocabulary at a time.
    workspace: fat_linear_cross_entropy_workspace_size(..., backward=True) bytes (None: allocated here),
    for one call at a time. Returns (dhidden bf16 [rows, dim] or None, dweight bf16 [vocab, dim] or
    None)."""
    r = (_calls or _load_calls()).lce_bwd(hidden, weight, target, lse, dloss, z_loss, logit_scale,
                                          grad_scale, want_dhidden, want_dweight, dhidden, dweight,
                                          workspace, _stream_arg(stream))
    if type(r) is int:
        raise FatAttnError(r, "fat_linear_cross_entropy_bwd")
    return r


def fat_paged_plan(ctx_lens, new_lens, free_pages, block_table, page_size: int, num_pages: int,
                   max_tokens: int, cu_seqlens_q=None, seqlens_k=None, positions=None, slots=None,
                   counts=None, stream=None):
    """The maps of a step in which request i (ctx_lens[i] cached tokens) brings new_lens[i] tokens:
    pages it lacks are taken from free_pages in request order and written to block_table (int32
    [n, width], in place). Returns (cu_seqlens_q [n + 1], seqlens_k [n], positions [max_tokens],
    slots [max_tokens], counts [2] = pages taken, tokens), all int32; tokens behind the last
    request get position 0 and slot -1. Given results must not lie over other arguments."""
    r = (_calls or _load_calls()).plan(ctx_lens, new_lens, free_pages, block_table, page_size,
                                       num_pages, max_tokens, cu_seqlens_q, seqlens_k, positions,
                                       slots, counts, _stream_arg(stream))
    if type(r) is int:
        raise FatAttnError(r, "fat_paged_plan")
    return r


def fat_rope_init(rotary_dim: int, base: float = 10000.0, interleaved: bool = True,
                  factor: float = 1.0, ramp=None, amplitude: float = 1.0) -> _Rope:
    """The rotation fat_rope_embed and fat_paged_append apply (made once, kept by the caller): the
    first rotary_dim channels of a head turn in pairs (2i, 2i + 1), or (i, i + rotary_dim / 2) when
    not interleaved. factor divides the frequencies; ramp = (low_turns, high_turns,
    original_length) keeps those that turn at least high_turns times over original_length and
    blends down to low_turns. amplitude multiplies the turned channels."""
    low, high, original = ramp if ramp is not None else (0.0, 0.0, 0.0)
    r = _Rope()
    rc = load().fat_rope_init(ctypes.byref(r), int(rotary_dim), int(bool(interleaved)),
                              float(base), float(factor), float(low), float(high),
                              float(original), float(amplitude))
    if rc != 0:
        raise FatAttnError(rc, "fat_rope_init")
    return r


def fat_rope_embed(x, positions, rope: _Rope, inverse: bool = False, out=None, stream=None):
    """Rotary embedding of bf16 rows x [T, H, d] (strided views are fine) at positions int32 [T];
    inverse=True applies the transpose, which takes the gradient of the result to the gradient of
    x. out may be x itself (in place). Returns out."""
    r = (_calls or _load_calls()).rope(x, positions, rope, inverse, out, _stream_arg(stream))
    if type(r) is int:
        raise FatAttnError(r, "fat_rope_embed")
    return r


def fat_paged_append(k, v, k_cache, v_cache, slots, q=None, positions=None, rope=None, q_out=None,
                     stream=None):
    """Write the rows k, v (bf16 [T, Hkv, d], strided views are fine) to their slots (int32 [T],
    page * page_size + offset; negative: dropped) of the caches (bf16 [pages, page_size, Hkv, d],
    any strides with a contiguous row, the same for both). With rope, k is turned at positions
    (int32 [T]) on the way, and q (bf16 [T, Hq, d]) too. Returns q_out (contiguous) or None."""
    r = (_calls or _load_calls()).append(k, v, k_cache, v_cache, slots, q, positions, rope, q_out,
                                         _stream_arg(stream))
    if type(r) is int:
        raise FatAttnError(r, "fat_paged_append")
    return r[0]


def fat_paged_attn_workspace_size(q, k_cache, cu_seqlens_q, max_seqlen_q: int,
                                  max_seqlen_k: int) -> int:
    """Workspace bytes of fat_paged_attn for these arguments on q's device, and for every call of
    fewer rows, requests, queries or keys: a buffer for the largest bounds serves all steps."""
    return (_calls or _load_calls()).attn_workspace(q, k_cache, cu_seqlens_q, max_seqlen_q,
                                                    max_seqlen_k)


def fat_paged_attn(q, k_cache, v_cache, block_table, cu_seqlens_q, seqlens_k, max_seqlen_q: int,
                   max_seqlen_k: int, bias_table=None, num_buckets: int = 0,
                   max_distance: int = 0, bidirectional: bool = True, alibi_slopes=None,
                   causal: bool = False, softmax_scale: float = 1.0, out=None, lse=None,
                   workspace=None, stream=None):
    """Attention of new tokens over a paged cache: q bf16 [Tq, Hq, d] packed by cu_seqlens_q (int32
    [n + 1]); request i's seqlens_k[i] keys and values lie in the pages block_table[i] (int32
    [n, width]) of the caches (bf16 [pages, page_size, Hkv, d], any strides with a contiguous row);
    its last query lines up with its last key. Bias, mask and scale as fat_xattn_fwd. workspace:
    fat_paged_attn_workspace_size bytes (None: allocated here), for one call at a time. Returns
    (out bf16 [Tq, Hq, d], lse fp32 [Hq, Tq])."""
    r = (_calls or _load_calls()).attn(q, k_cache, v_cache, block_table, cu_seqlens_q, seqlens_k,
                                       max_seqlen_q, max_seqlen_k, bias_table, num_buckets,
                                       max_distance, bidirectional, alibi_slopes, causal,
                                       softmax_scale, out, lse, workspace, _stream_arg(stream))
    if type(r) is int:
        raise FatAttnError(r, "fat_paged_attn")
    return r


def fat_paged_tree_plan(parents, cu_seqlens_q, seqlens_k, max_seqlen_q: int, positions=None,
                        tree_mask=None, stream=None):
    """The maps of a step whose new tokens are trees of drafted tokens: parents int32 [T], of each
    node the index within its request of the earlier node that it follows (-1: the cached context).
    Returns (positions int32 [T] = seqlens_k - nodes + depth, tree_mask int32 [T, words]: the bits of
    the node's path). Rows behind the last request get 0."""
    r = (_calls or _load_calls()).tree_plan(parents, cu_seqlens_q, seqlens_k, max_seqlen_q, positions,
                                            tree_mask, _stream_arg(stream))
    if type(r) is int:
        raise FatAttnError(r, "fat_paged_tree_plan")
    return r


def fat_paged_tree_attn(q, k_cache, v_cache, block_table, cu_seqlens_q, seqlens_k, positions,
                        tree_mask, max_seqlen_q: int, max_seqlen_k: int, bias_table=None,
                        num_buckets: int = 0, max_distance: int = 0, bidirectional: bool = True,
                        alibi_slopes=None, softmax_scale: float = 1.0, out=None, lse=None,
                        workspace=None, stream=None):
    """fat_paged_attn for trees of drafted tokens (appended first): a query sees the keys before its
    request's first query and, of the request's own, those whose bit is set in its row of tree_mask
    (int32 [Tq, words], any pattern); biases go by positions (int32 [Tq]). fat_paged_tree_plan makes
    both. workspace: fat_paged_attn_workspace_size bytes (None: allocated here), for one call at a
    time. Returns (out bf16 [Tq, Hq, d], lse fp32 [Hq, Tq])."""
    r = (_calls or _load_calls()).tree_attn(q, k_cache, v_cache, block_table, cu_seqlens_q, seqlens_k,
                                            positions, tree_mask, max_seqlen_q, max_seqlen_k,
                                            bias_table, num_buckets, max_distance, bidirectional,
                                            alibi_slopes, softmax_scale, out, lse, workspace,
                                            _stream_arg(stream))
    if type(r) is int:
        raise FatAttnError(r, "fat_paged_tree_attn")
    return r


def fat_attn_get_device_error(stream=None, device=None) -> int:
    """Synchronise, read and clear the device error word; returns its bits (0 = no error)."""
    lib = load()
    bits = ctypes.c_int(0)
    rc = lib.fat_attn_get_device_error(_stream_ptr(stream, device), ctypes.byref(bits))
    if rc not in (0, -6):
        raise FatAttnError(rc, "fat_attn_get_device_error")
    return int(bits.value)


def fat_attn_strerror(code: int) -> str:
    return load().fat_attn_strerror(int(code)).decode()


def fat_attn_bucket_thresholds(num_buckets: int, max_distance: int, bidirectional: bool):
    """Host-side thresholds the kernels compare distances with: (thresholds list, saturation)."""
    lib = load()
    arr = (ctypes.c_int32 * 64)()
    cnt, sat = ctypes.c_int(0), ctypes.c_int(0)
    rc = lib.fat_attn_bucket_thresholds(int(num_buckets), int(max_distance),
                                        int(bool(bidirectional)), arr, ctypes.byref(cnt),
                                        ctypes.byref(sat))
    if rc != 0:
        raise FatAttnError(rc, "fat_attn_bucket_thresholds")
    return list(arr[: cnt.value]), int(sat.value)


def fat_attn_debug_buckets(delta_lo: int, n: int, num_buckets: int, max_distance: int,
                           bidirectional: bool, out=None, stream=None, device="cuda"):
    """Device-side T5 bucket ids for delta_lo .. delta_lo+n-1 (int32 CUDA tensor)."""
    import torch
    lib = load()
    if out is None:
        out = torch.empty(n, dtype=torch.int32, device=device)
    with _on(out.device):
        rc = lib.fat_attn_debug_buckets(int(delta_lo), int(n), int(num_buckets), int(max_distance),
                                        int(bool(bidirectional)), _ptr(out),
                                        _stream_ptr(stream, out.device))
    if rc != 0:
        raise FatAttnError(rc, "fat_attn_debug_buckets")
    return out


def fat_attn_debug_set_watchdog(timeout_ns: int = 0, flags: int = 0) -> None:
    load().fat_attn_debug_set_watchdog(int(timeout_ns), int(flags))
