"""Python binding of libsdpa.so, the fused SDPA library for one GB300 GPU.

The functions carry the C ABI's names (include/sdpa.h) and only marshal
arguments: torch supplies device memory and the current CUDA stream, and every
step of the computation runs in the library's CUDA kernels. There is no other
implementation behind these calls: if libsdpa.so is missing, or the tensors
are not CUDA tensors, the call raises.

Layouts: "bshd" [B,S,H,D], "sbhd" [S,B,H,D], "thd" [T,H,D] (+ cu_seqlens).
Masks: "none", "causal" (top-left), "causal_br" (bottom-right).
V (and O, dO) may be narrower than Q/K for the forward's 192/128 pair; the
binding reads that width from v. Tensor shapes, dtypes and devices are checked
against each other from metadata before the library is called.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os
import threading

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libsdpa.so")
CHECKED_LIB_PATH = os.path.join(PKG, "libsdpa_checked.so")  # the address-checked testing build

LAYOUTS = {"bshd": 0, "sbhd": 1, "thd": 2}
MASKS = {"none": 0, "causal": 1, "causal_br": 2}
STATUS = {0: "SDPA_OK", 1: "SDPA_ERR_INVALID_ARG", 2: "SDPA_ERR_UNSUPPORTED", 3: "SDPA_ERR_ALIGNMENT",
          4: "SDPA_ERR_OVERLAP", 5: "SDPA_ERR_WORKSPACE_TOO_SMALL", 6: "SDPA_ERR_BAD_SEQLENS",
          7: "SDPA_ERR_TIMEOUT", 8: "SDPA_ERR_CUDA", 9: "SDPA_ERR_ADDRESS",
          10: "SDPA_ERR_BAD_INDEX"}
EXPORTS = ("sdpa_fwd_workspace_size", "sdpa_bwd_workspace_size", "sdpa_check_problem", "sdpa_fwd", "sdpa_bwd",
           "sdpa_get_device_error", "sdpa_error_string", "sdpa_last_launch_count", "sdpa_profile_begin",
           "sdpa_profile_end", "sdpa_bwd_noalloc", "sdpa_selftest_bounded_wait", "sdpa_merge",
           "sdpa_fwd_fp8_workspace_size", "sdpa_fwd_fp8", "sdpa_debug_set_max_ctas", "sdpa_debug_address_report",
           "sdpa_debug_address_shrink", "sdpa_qk_norm_rope", "sdpa_qk_norm_rope_bwd_workspace_size",
           "sdpa_qk_norm_rope_bwd", "sdpa_check_paged", "sdpa_paged_append", "sdpa_paged_fwd_workspace_size",
           "sdpa_paged_fwd")
NOALLOC_MAX_BYTES = 32 << 20  # SDPA_BWD_NOALLOC_MAX_BYTES
PAGED_WORKSPACE_MAX = 256 << 20  # SDPA_PAGED_WORKSPACE_MAX
PAGED_KEYS_MAX = 1 << 30  # the longest kv_len that the library serves
KERNEL_KINDS = ("fwd", "bwd", "preprocess", "dq_finalize", "guard", "merge", "bwd_dq", "v_transpose",
                "norm_rope", "append", "paged")


class SdpaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)} ({error_string(status)})")


class MergeProblem(ctypes.Structure):
    """sdpa_merge_problem (include/sdpa.h)."""
    _fields_ = [("dtype", ctypes.c_int), ("items", ctypes.c_longlong), ("head_dim", ctypes.c_int),
                ("n_parts", ctypes.c_int)]


class NormRopeProblem(ctypes.Structure):
    """sdpa_norm_rope_problem (include/sdpa.h)."""
    _fields_ = [(n, ctypes.c_int) for n in ("dtype", "num_heads_q", "num_heads_kv", "head_dim", "rotary_dim",
                                            "interleaved")] + [("eps", ctypes.c_float),
                                                               ("max_positions", ctypes.c_int)] + [
        (n, ctypes.c_longlong) for n in ("rows", "q_stride", "k_stride", "dq_stride", "dk_stride")]


class PagedProblem(ctypes.Structure):
    """sdpa_paged_problem (include/sdpa.h)."""
    _fields_ = [(n, ctypes.c_int) for n in ("dtype", "batch", "num_heads_q", "num_heads_kv", "head_dim", "head_dim_v",
                                            "total_q", "seqlen_q", "seqlen_kv", "page_size", "num_pages", "max_pages",
                                            "mask_type", "window_left")] + [("softmax_scale", ctypes.c_float)] + [
        (n, ctypes.c_longlong) for n in ("table_stride", "k_page_stride", "k_slot_stride", "k_head_stride",
                                         "v_page_stride", "v_slot_stride", "v_head_stride", "q_stride", "k_stride",
                                         "v_stride")]


class Problem(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("layout", "dtype", "mask_type", "batch", "seqlen_q", "seqlen_kv",
                                            "total_q", "total_kv", "num_heads_q", "num_heads_kv", "head_dim",
                                            "window_left", "window_right")] + [("softmax_scale", ctypes.c_float),
                                                                               ("deterministic", ctypes.c_int),
                                                                               ("head_dim_v", ctypes.c_int),
                                                                               ("kv_chunk", ctypes.c_int)]


_lock = threading.Lock()
_libs = {}
_active = LIB_PATH


def _load(path):
    if path not in _libs:
        if not os.path.exists(path):
            raise ImportError(f"{path} is missing: run scaled_dot_product_02_gb300/build.py "
                              "(there is no fallback implementation)")
        L = ctypes.CDLL(path)
        vp, pp = ctypes.c_void_p, ctypes.POINTER(Problem)
        L.sdpa_fwd_workspace_size.argtypes = [pp]
        L.sdpa_fwd_workspace_size.restype = ctypes.c_size_t
        L.sdpa_bwd_workspace_size.argtypes = [pp]
        L.sdpa_bwd_workspace_size.restype = ctypes.c_size_t
        L.sdpa_check_problem.argtypes = [pp]
        L.sdpa_fwd.argtypes = [pp, vp, vp, vp, vp, vp, vp, vp, vp, ctypes.c_size_t, vp]
        L.sdpa_bwd.argtypes = [pp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, ctypes.c_size_t, vp]
        L.sdpa_get_device_error.argtypes = [vp]
        L.sdpa_error_string.argtypes = [ctypes.c_int]
        L.sdpa_error_string.restype = ctypes.c_char_p
        L.sdpa_last_launch_count.restype = ctypes.c_int
        L.sdpa_selftest_bounded_wait.argtypes = [ctypes.c_uint, vp]
        L.sdpa_debug_set_max_ctas.argtypes = [ctypes.c_int]
        u64p = ctypes.POINTER(ctypes.c_ulonglong)
        L.sdpa_debug_address_report.argtypes = [u64p, u64p, u64p]
        L.sdpa_debug_address_shrink.argtypes = [ctypes.c_longlong]
        L.sdpa_bwd_noalloc.argtypes = [pp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
        L.sdpa_merge.argtypes = [ctypes.POINTER(MergeProblem), vp, vp, vp, vp, vp]
        L.sdpa_profile_end.argtypes = [ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_int),
                                       ctypes.c_int]
        L.sdpa_fwd_fp8_workspace_size.argtypes = [pp]
        L.sdpa_fwd_fp8_workspace_size.restype = ctypes.c_size_t
        fl = ctypes.c_float
        L.sdpa_fwd_fp8.argtypes = [pp, vp, vp, vp, fl, fl, fl, vp, vp, vp, vp, vp, ctypes.c_size_t, vp]
        npp, ppp = ctypes.POINTER(NormRopeProblem), ctypes.POINTER(PagedProblem)
        L.sdpa_qk_norm_rope.argtypes = [npp] + [vp] * 9
        L.sdpa_qk_norm_rope_bwd_workspace_size.argtypes = [npp]
        L.sdpa_qk_norm_rope_bwd_workspace_size.restype = ctypes.c_size_t
        L.sdpa_qk_norm_rope_bwd.argtypes = [npp] + [vp] * 13 + [ctypes.c_size_t, vp]
        L.sdpa_check_paged.argtypes = [ppp]
        L.sdpa_paged_append.argtypes = [ppp, npp] + [vp] * 14
        L.sdpa_paged_fwd_workspace_size.argtypes = [ppp]
        L.sdpa_paged_fwd_workspace_size.restype = ctypes.c_size_t
        L.sdpa_paged_fwd.argtypes = [ppp] + [vp] * 9 + [ctypes.c_size_t, vp]
        _libs[path] = L
    return _libs[path]


def lib():
    """The loaded library every call goes through: libsdpa.so, or
    libsdpa_checked.so inside `address_checked()` (build them first with
    scaled_dot_product_02_gb300.build)."""
    with _lock:
        return _load(_active)


@contextlib.contextmanager
def address_checked():
    """Testing aid: route the calls made inside the block through
    libsdpa_checked.so, whose kernels test every computed global access
    against the call's buffers (sdpa_debug_address_report in include/sdpa.h).
    Both libraries stay loaded; each keeps its own device error word."""
    global _active
    with _lock:
        prev, _active = _active, CHECKED_LIB_PATH
        _load(CHECKED_LIB_PATH)
    try:
        yield
    finally:
        with _lock:
            _active = prev


def sdpa_debug_address_report():
    """(violations, first address, its size) since the last report, then
    cleared (synchronises the device). Address-checked library only."""
    v, a, n = ctypes.c_ulonglong(0), ctypes.c_ulonglong(0), ctypes.c_ulonglong(0)
    rc = lib().sdpa_debug_address_report(ctypes.byref(v), ctypes.byref(a), ctypes.byref(n))
    if rc:
        raise SdpaError(rc, "sdpa_debug_address_report")
    return v.value, a.value, n.value


def sdpa_debug_address_shrink(nbytes: int) -> None:
    """Pull the end of every extent registered from now on in by nbytes (0
    restores them). Address-checked library only."""
    rc = lib().sdpa_debug_address_shrink(int(nbytes))
    if rc:
        raise SdpaError(rc, "sdpa_debug_address_shrink")


def error_string(status: int) -> str:
    return lib().sdpa_error_string(int(status)).decode()


sdpa_error_string = error_string


def make_problem(q, k, *, layout="bshd", mask="none", window=(-1, -1), scale=None, dtype=None, batch=None,
                 max_seqlen_q=None, max_seqlen_kv=None, deterministic=False, head_dim_v=0, kv_chunk=0) -> Problem:
    """sdpa_problem from tensor shapes (no device access). head_dim_v: the
    width of V and O rows (0 = Q/K's head_dim). kv_chunk: key positions per
    chunk of the head_dim 256/512 backward (a multiple of 128; 0 = the
    library's choice)."""
    import torch

    if dtype is None:
        dtype = {torch.bfloat16: 0, torch.float16: 1}.get(q.dtype, -1)
    d = q.shape[-1]
    p = Problem()
    p.layout, p.dtype, p.mask_type = LAYOUTS[layout], dtype, MASKS[mask]
    if layout == "bshd":
        p.batch, p.seqlen_q, p.num_heads_q = q.shape[0], q.shape[1], q.shape[2]
        p.seqlen_kv, p.num_heads_kv = k.shape[1], k.shape[2]
    elif layout == "sbhd":
        p.seqlen_q, p.batch, p.num_heads_q = q.shape[0], q.shape[1], q.shape[2]
        p.seqlen_kv, p.num_heads_kv = k.shape[0], k.shape[2]
    else:
        if batch is None or max_seqlen_q is None or max_seqlen_kv is None:
            raise ValueError("thd needs batch, max_seqlen_q and max_seqlen_kv")
        p.batch, p.seqlen_q, p.seqlen_kv = batch, max_seqlen_q, max_seqlen_kv
        p.total_q, p.total_kv = q.shape[0], k.shape[0]
        p.num_heads_q, p.num_heads_kv = q.shape[1], k.shape[1]
    p.head_dim = d
    p.window_left, p.window_right = int(window[0]), int(window[1])
    p.softmax_scale = float(scale if scale is not None else d ** -0.5)
    p.deterministic = int(bool(deterministic))
    p.head_dim_v = int(head_dim_v)
    p.kv_chunk = int(kv_chunk)
    return p


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    import torch

    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check_cuda(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("sdpa tensors must be CUDA tensors (there is no CPU implementation)")
        if t is not None and not t.is_contiguous():
            raise ValueError("sdpa tensors must be contiguous in their layout")


def _validate(layout, q, k, v, *, o=None, lse=None, dout=None, dq=None, dk=None, dv=None, cu_q=None, cu_kv=None):
    """Shapes, dtypes and devices of one call's tensors, from their metadata
    alone (no device access, no synchronisation). The C ABI receives bare
    pointers and sizes taken from q and k, so a tensor smaller than the
    problem it is part of would let the kernels read or write past its end:
    such calls are refused here with ValueError."""
    import torch

    if q.dtype not in (torch.bfloat16, torch.float16):
        raise ValueError(f"q must be bfloat16 or float16, got {q.dtype}")
    rank = 3 if layout == "thd" else 4
    for name, t in (("q", q), ("k", k), ("v", v)):
        if t.dim() != rank:
            raise ValueError(f"{name} must have {rank} dimensions in layout {layout}, got {tuple(t.shape)}")
        if t.dtype != q.dtype or t.device != q.device:
            raise ValueError(f"{name} must have q's dtype and device ({q.dtype}, {q.device})")
    if k.shape[-1] != q.shape[-1]:
        raise ValueError(f"q and k must share head_dim, got {q.shape[-1]} and {k.shape[-1]}")
    if tuple(k.shape[:-1]) != tuple(v.shape[:-1]):
        raise ValueError(f"k and v must agree on every dimension but the last, got {tuple(k.shape)} and "
                         f"{tuple(v.shape)}")
    batch_dim = {"bshd": 0, "sbhd": 1}.get(layout)
    if batch_dim is not None and q.shape[batch_dim] != k.shape[batch_dim]:
        raise ValueError(f"q and k must have the same batch size, got {q.shape[batch_dim]} and {k.shape[batch_dim]}")
    o_shape = tuple(q.shape[:-1]) + (v.shape[-1],)
    rows_q = q.numel() // max(1, q.shape[-1] * q.shape[-2])
    for name, t, shape, dtype in (("o", o, o_shape, q.dtype), ("dout", dout, o_shape, q.dtype),
                                  ("dq", dq, tuple(q.shape), q.dtype), ("dk", dk, tuple(k.shape), q.dtype),
                                  ("dv", dv, tuple(v.shape), q.dtype),
                                  ("lse", lse, (rows_q, q.shape[-2]), torch.float32)):
        if t is None:
            continue
        if tuple(t.shape) != shape or t.dtype != dtype or t.device != q.device:
            raise ValueError(f"{name} must be {dtype} of shape {shape} on {q.device}, got {t.dtype} "
                             f"{tuple(t.shape)} on {t.device}")
    for name, t in (("cu_seqlens_q", cu_q), ("cu_seqlens_kv", cu_kv)):
        if t is None:
            continue
        if t.dtype != torch.int32 or t.dim() != 1 or t.numel() < 1 or t.device != q.device:
            raise ValueError(f"{name} must be a 1-D int32 tensor of batch + 1 entries on {q.device}")
    if cu_q is not None and cu_kv is not None and cu_q.numel() != cu_kv.numel():
        raise ValueError("cu_seqlens_q and cu_seqlens_kv must have the same number of entries")


def sdpa_check_problem(p: Problem) -> int:
    return int(lib().sdpa_check_problem(ctypes.byref(p)))


def sdpa_fwd_workspace_size(p: Problem) -> int:
    return int(lib().sdpa_fwd_workspace_size(ctypes.byref(p)))


def sdpa_bwd_workspace_size(p: Problem) -> int:
    return int(lib().sdpa_bwd_workspace_size(ctypes.byref(p)))


def sdpa_fwd(q, k, v, *, layout="bshd", mask="none", window=(-1, -1), scale=None, cu_seqlens_q=None,
             cu_seqlens_kv=None, max_seqlen_q=None, max_seqlen_kv=None, out=None, lse=None, workspace=None,
             stream=None):
    """Forward. Returns (o, lse); o has Q's shape with V's last dimension,
    lse is float32 [rows_q, Hq] token-major."""
    import torch

    batch = None if cu_seqlens_q is None else cu_seqlens_q.numel() - 1
    p = make_problem(q, k, layout=layout, mask=mask, window=window, scale=scale, batch=batch,
                     max_seqlen_q=max_seqlen_q, max_seqlen_kv=max_seqlen_kv, head_dim_v=v.shape[-1])
    rows_q = q.numel() // (q.shape[-1] * q.shape[-2])
    if out is None:
        out = torch.empty(tuple(q.shape[:-1]) + (v.shape[-1],), dtype=q.dtype, device=q.device)
    if lse is None:
        lse = torch.empty((rows_q, q.shape[-2]), dtype=torch.float32, device=q.device)
    _validate(layout, q, k, v, o=out, lse=lse, cu_q=cu_seqlens_q, cu_kv=cu_seqlens_kv)
    need = sdpa_fwd_workspace_size(p)
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    _check_cuda(q, k, v, out, lse, cu_seqlens_q, cu_seqlens_kv, workspace)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = lib().sdpa_fwd(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(cu_seqlens_q),
                        _ptr(cu_seqlens_kv), _ptr(workspace), ws_bytes, _stream(stream))
    if rc:
        raise SdpaError(rc, "sdpa_fwd")
    return out, lse


def sdpa_bwd(q, k, v, o, lse, dout, *, layout="bshd", mask="none", window=(-1, -1), scale=None,
             cu_seqlens_q=None, cu_seqlens_kv=None, max_seqlen_q=None, max_seqlen_kv=None, dq=None, dk=None,
             dv=None, workspace=None, stream=None, deterministic=False, kv_chunk=0):
    """Backward. Returns (dq, dk, dv). deterministic=True makes every
    gradient bitwise reproducible run to run (see sdpa_problem.deterministic);
    kv_chunk sets sdpa_problem.kv_chunk (head_dim 256/512)."""
    import torch

    batch = None if cu_seqlens_q is None else cu_seqlens_q.numel() - 1
    p = make_problem(q, k, layout=layout, mask=mask, window=window, scale=scale, batch=batch,
                     max_seqlen_q=max_seqlen_q, max_seqlen_kv=max_seqlen_kv, deterministic=deterministic,
                     head_dim_v=v.shape[-1], kv_chunk=kv_chunk)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    _validate(layout, q, k, v, o=o, lse=lse, dout=dout, dq=dq, dk=dk, dv=dv, cu_q=cu_seqlens_q, cu_kv=cu_seqlens_kv)
    need = sdpa_bwd_workspace_size(p)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    _check_cuda(q, k, v, o, lse, dout, dq, dk, dv, cu_seqlens_q, cu_seqlens_kv, workspace)
    ws_bytes = workspace.numel() * workspace.element_size()
    rc = lib().sdpa_bwd(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout), _ptr(dq),
                        _ptr(dk), _ptr(dv), _ptr(cu_seqlens_q), _ptr(cu_seqlens_kv), _ptr(workspace), ws_bytes,
                        _stream(stream))
    if rc:
        raise SdpaError(rc, "sdpa_bwd")
    return dq, dk, dv


def sdpa_bwd_noalloc(q, k, v, o, lse, dout, *, layout="bshd", mask="none", window=(-1, -1), scale=None,
                     cu_seqlens_q=None, cu_seqlens_kv=None, max_seqlen_q=None, max_seqlen_kv=None, dq=None,
                     dk=None, dv=None, stream=None, deterministic=False, kv_chunk=0):
    """Backward without a workspace: the library's static scratch array is
    used instead (for callers that cannot allocate device memory; problems
    needing more than NOALLOC_MAX_BYTES of scratch are rejected). Calls that
    overlap on the GPU race on that array. Returns (dq, dk, dv); pass dq/dk/dv
    to avoid torch allocating them here."""
    import torch

    batch = None if cu_seqlens_q is None else cu_seqlens_q.numel() - 1
    p = make_problem(q, k, layout=layout, mask=mask, window=window, scale=scale, batch=batch,
                     max_seqlen_q=max_seqlen_q, max_seqlen_kv=max_seqlen_kv, deterministic=deterministic,
                     head_dim_v=v.shape[-1], kv_chunk=kv_chunk)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    _validate(layout, q, k, v, o=o, lse=lse, dout=dout, dq=dq, dk=dk, dv=dv, cu_q=cu_seqlens_q, cu_kv=cu_seqlens_kv)
    _check_cuda(q, k, v, o, lse, dout, dq, dk, dv, cu_seqlens_q, cu_seqlens_kv)
    rc = lib().sdpa_bwd_noalloc(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout),
                                _ptr(dq), _ptr(dk), _ptr(dv), _ptr(cu_seqlens_q), _ptr(cu_seqlens_kv),
                                _stream(stream))
    if rc:
        raise SdpaError(rc, "sdpa_bwd_noalloc")
    return dq, dk, dv


def sdpa_fwd_fp8_workspace_size(p: Problem) -> int:
    return int(lib().sdpa_fwd_fp8_workspace_size(ctypes.byref(p)))


def sdpa_fwd_fp8(q8, k8, v8, *, descale=(1.0, 1.0, 1.0), layout="bshd", mask="none", window=(-1, -1), scale=None,
                 cu_seqlens_q=None, cu_seqlens_kv=None, max_seqlen_q=None, max_seqlen_kv=None, out_dtype=None,
                 out=None, lse=None, workspace=None, stream=None):
    """FP8 E4M3 forward (head_dim 128 or 256). q8, k8, v8: torch.uint8 codes or
    torch.float8_e4m3fn tensors in `layout`; descale = (d_q, d_k, d_v), the
    per-tensor factors that turn codes into values. The softmax output is
    stored as E4M3(exp(S - m) * 448), m the row's final maximum, and O divides
    by 448 times the row sum (see sdpa_fwd_fp8 in include/sdpa.h). Returns (o, lse): o in out_dtype (default bfloat16) with
    q8's shape, lse float32 [rows_q, Hq]."""
    import torch

    f8 = getattr(torch, "float8_e4m3fn", None)
    for name, t in (("q8", q8), ("k8", k8), ("v8", v8)):
        if t.dtype not in (torch.uint8, f8):
            raise ValueError(f"{name} must hold E4M3 codes (torch.uint8 or torch.float8_e4m3fn), got {t.dtype}")
        if t.device != q8.device:
            raise ValueError(f"{name} must be on q8's device")
    out_dtype = torch.bfloat16 if out_dtype is None else out_dtype
    if out_dtype not in (torch.bfloat16, torch.float16):
        raise ValueError("out_dtype must be bfloat16 or float16")
    rank = 3 if layout == "thd" else 4
    if any(t.dim() != rank for t in (q8, k8, v8)):
        raise ValueError(f"q8, k8, v8 must have {rank} dimensions in layout {layout}")
    if tuple(k8.shape) != tuple(v8.shape) or k8.shape[-1] != q8.shape[-1]:
        raise ValueError("k8 and v8 must have the same shape, and the same head_dim as q8")
    batch = None if cu_seqlens_q is None else cu_seqlens_q.numel() - 1
    p = make_problem(q8, k8, layout=layout, mask=mask, window=window, scale=scale, batch=batch,
                     dtype={torch.bfloat16: 0, torch.float16: 1}[out_dtype], max_seqlen_q=max_seqlen_q,
                     max_seqlen_kv=max_seqlen_kv)
    rows_q = q8.numel() // (q8.shape[-1] * q8.shape[-2])
    if out is None:
        out = torch.empty(tuple(q8.shape), dtype=out_dtype, device=q8.device)
    if lse is None:
        lse = torch.empty((rows_q, q8.shape[-2]), dtype=torch.float32, device=q8.device)
    if tuple(out.shape) != tuple(q8.shape) or out.dtype != out_dtype or tuple(lse.shape) != (rows_q, q8.shape[-2]) \
            or lse.dtype != torch.float32:
        raise ValueError("out must have q8's shape in out_dtype and lse float32 [rows_q, Hq]")
    for name, t in (("cu_seqlens_q", cu_seqlens_q), ("cu_seqlens_kv", cu_seqlens_kv)):
        if t is not None and (t.dtype != torch.int32 or t.dim() != 1 or t.device != q8.device):
            raise ValueError(f"{name} must be a 1-D int32 tensor on q8's device")
    need = sdpa_fwd_fp8_workspace_size(p)
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=q8.device)
    _check_cuda(q8, k8, v8, out, lse, cu_seqlens_q, cu_seqlens_kv, workspace)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = lib().sdpa_fwd_fp8(ctypes.byref(p), _ptr(q8), _ptr(k8), _ptr(v8), float(descale[0]), float(descale[1]),
                            float(descale[2]), _ptr(out), _ptr(lse), _ptr(cu_seqlens_q), _ptr(cu_seqlens_kv),
                            _ptr(workspace), ws_bytes, _stream(stream))
    if rc:
        raise SdpaError(rc, "sdpa_fwd_fp8")
    return out, lse


def sdpa_get_device_error(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device error word."""
    return int(lib().sdpa_get_device_error(_stream(stream)))


def sdpa_debug_set_max_ctas(max_ctas: int) -> None:
    """Testing aid: cap the CTAs of every attention kernel launch (0 = no
    cap). See sdpa_debug_set_max_ctas in include/sdpa.h."""
    rc = lib().sdpa_debug_set_max_ctas(int(max_ctas))
    if rc:
        raise SdpaError(rc, "sdpa_debug_set_max_ctas")


def sdpa_last_launch_count() -> int:
    return int(lib().sdpa_last_launch_count())


def sdpa_profile_begin() -> None:
    """Start recording CUDA events around every kernel this thread's calls launch."""
    lib().sdpa_profile_begin()


def sdpa_profile_end() -> dict:
    """Stop recording; returns {kind: (total_ms, launches)} (synchronises)."""
    n = len(KERNEL_KINDS)
    ms = (ctypes.c_double * n)()
    cnt = (ctypes.c_int * n)()
    rc = lib().sdpa_profile_end(ms, cnt, n)
    if rc:
        raise SdpaError(rc, "sdpa_profile_end")
    return {k: (ms[i], cnt[i]) for i, k in enumerate(KERNEL_KINDS)}


def sdpa_merge(o_parts, lse_parts, *, out=None, lse=None, stream=None):
    """Log-sum-exp merge of partial results over a split of the keys.

    o_parts: [P, ..., H, D] (bf16/fp16, the forward's O over P key blocks,
    stacked); lse_parts: fp32 [P, rows, H] (the forward's LSE). Returns
    (o [..., H, D], lse [rows, H]).
    """
    import torch

    n = o_parts.shape[0]
    d = o_parts.shape[-1]
    items = o_parts[0].numel() // d
    if out is None:
        out = torch.empty(o_parts.shape[1:], dtype=o_parts.dtype, device=o_parts.device)
    if lse is None:
        lse = torch.empty(lse_parts.shape[1:], dtype=torch.float32, device=o_parts.device)
    if lse_parts.dtype != torch.float32 or lse_parts.numel() != n * items or lse.numel() != items:
        raise ValueError("lse_parts must be float32 [P, rows, H] matching o_parts")
    if lse.dtype != torch.float32 or out.dtype != o_parts.dtype or out.numel() != items * d:
        raise ValueError("out must have o_parts' dtype and o_parts[0]'s size, lse must be float32 [rows, H]")
    if len({t.device for t in (o_parts, lse_parts, out, lse)}) != 1:
        raise ValueError("sdpa_merge tensors must be on one device")
    for t in (o_parts, lse_parts, out, lse):
        if not t.is_contiguous():
            raise ValueError("sdpa_merge needs contiguous tensors")
    _check_cuda(o_parts, lse_parts, out, lse)
    dt = {torch.bfloat16: 0, torch.float16: 1}.get(o_parts.dtype)
    if dt is None:
        raise ValueError("o_parts must be bf16 or fp16")
    p = MergeProblem(dt, items, d, n)
    rc = lib().sdpa_merge(ctypes.byref(p), _ptr(o_parts), _ptr(lse_parts), _ptr(out), _ptr(lse), _stream(stream))
    if rc:
        raise SdpaError(rc, "sdpa_merge")
    return out, lse

# ---------------------------------------------------------------- norms, rotation, paged cache
# The checks below depend on the tensors' metadata alone, so they are made once
# per combination of it (_meta is the key) and kept, with the problem struct that
# they lead to: a decoding step repeats its calls with the same shapes, and the
# checks took longer than the kernels. Nothing is kept by address or contents
# (scalars are turned into numbers before: a tensor's key would be its identity).
_torch_state = {}  # what the calls take from torch, looked up once
_PLANS = 512       # combinations kept per entry point


def _torch():
    if not _torch_state:
        import torch

        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        like = functools.partial(torch.empty_like, memory_format=torch.contiguous_format)  # quicker than new_empty
        _torch_state.update(torch=torch, like=like, codes={torch.bfloat16: 0, torch.float16: 1}, f32=torch.float32, i32=torch.int32,
                            raw=raw or (lambda index: torch.cuda.current_stream(index).cuda_stream))
    return _torch_state


def _meta(t):
    return None if t is None else (t.shape, t.stride(), t.dtype, t.device)


def _dtype_code(dtype, name):
    code = _torch()["codes"].get(dtype)
    if code is None:
        raise ValueError(f"{name} must be bfloat16 or float16, got {dtype}")
    return code


def _on(stream, entry, args):
    """entry(**args) with `stream` current, as torch's own operators run on a
    stream: the workspace and the outputs are allocated on it (from the current
    stream's memory the workspace would be handed out again while the kernels
    use it). Memory of other streams that the call uses, and what it returns to
    the calling stream, is kept until both are done with it."""
    torch = _torch()["torch"]
    tensors = [t for t in args.values() if isinstance(t, torch.Tensor)]
    for t in tensors:
        if t.device != stream.device:
            raise ValueError(f"the stream is on {stream.device}, the tensors on {t.device}")
    caller = torch.cuda.current_stream(stream.device)
    with torch.cuda.stream(stream):
        got = entry(**{**args, "stream": None})
    for t in tensors:
        t.record_stream(stream)
    for t in got if isinstance(got, tuple) else (got,):
        if t is not None:
            t.record_stream(caller)
    return got


def _launch(name, device, *args):
    """Call the entry point `name` with the raw handle of the device's current
    stream appended and `device` current: it launches on the calling thread's
    current device, so tensors of another one select theirs for the call."""
    torch = _torch_state["torch"]
    index = device.index
    raw = _torch_state["raw"](index)
    if index == torch.cuda.current_device():
        rc = getattr(lib(), name)(*args, raw)
    else:
        with torch.cuda.device(device):
            rc = getattr(lib(), name)(*args, raw)
    if rc:
        raise SdpaError(rc, name)


def _refuse_cpu(t):
    if not t.is_cuda:
        raise ValueError("sdpa tensors must be CUDA tensors (there is no CPU implementation)")


def _addr(t):
    return None if t is None else t.data_ptr()


def _contiguous(shape, st):
    step = 1
    for n, s in zip(reversed(shape), reversed(st)):
        if n != 1 and s != step:
            return 0 in shape
        step *= n
    return True


def _expect(name, meta, shape, dtype, device):
    got, st, got_dtype, got_device = meta
    if got_dtype is not dtype or got_device != device or tuple(got) != tuple(shape) or not _contiguous(got, st):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}, got "
                         f"{got_dtype} {tuple(got)} on {got_device}")


def _rows_of_heads(name, meta, like=None):
    """(rows, heads, head_dim, elements between rows) of [..., H, D] whose
    leading dimensions are one evenly spaced row index (contiguous, or a slice
    of a fused projection's output) and whose heads are contiguous."""
    shape, st, dtype, device = meta
    if like is not None and (dtype is not like[2] or device != like[3]):
        raise ValueError(f"{name} must have dtype {like[2]} on {like[3]}, got {dtype} on {device}")
    if len(shape) < 3:
        raise ValueError(f"{name} must have at least 3 dimensions [..., heads, head_dim], got {tuple(shape)}")
    h, d = shape[-2], shape[-1]
    rows, step, spaced = 1, None, st[-1] == 1 and (st[-2] == d or h == 1)
    for n, s in zip(reversed(shape[:-2]), reversed(st[:-2])):
        if n != 1:
            if step is None:
                step = s
                spaced = spaced and s >= h * d  # broadcast rows too: the C entry takes a stride of zero for contiguous
            elif s != rows * step:
                spaced = False
            rows *= n
    if rows and not spaced:
        raise ValueError(f"{name} must hold contiguous heads in evenly spaced rows, got shape {tuple(shape)} and "
                         f"strides {tuple(st)}")
    return rows, h, d, step if step is not None and rows else h * d


def _rotation(q, d, rows, q_weight, k_weight, cos_sin, positions, needs_positions):
    """(max_positions, rotary_dim) of the table; checks the weights, the table and the positions."""
    _, _, dtype, dev = q
    _expect("q_weight", q_weight, (d,), dtype, dev)
    _expect("k_weight", k_weight, (d,), dtype, dev)
    if cos_sin is None:
        return 0, 0
    shape = cos_sin[0]
    if len(shape) != 2:
        raise ValueError(f"cos_sin must be [positions, rotary_dim], got {tuple(shape)}")
    _expect("cos_sin", cos_sin, shape, _torch()["f32"], dev)
    if positions is not None:
        n = 1
        for x in positions[0]:
            n *= x
        if n != rows:
            raise ValueError(f"positions must have one entry per token ({rows}), got {tuple(positions[0])}")
        _expect("positions", positions, positions[0], _torch()["i32"], dev)
    elif needs_positions and shape[1]:
        raise ValueError("a rotation needs the tokens' positions")
    return shape


@functools.lru_cache(maxsize=_PLANS)
def _norm_rope_plan(q, k, q_weight, k_weight, cos_sin, positions, q_out, k_out, dq, dk, dq_out, dk_out, dq_weight,
                    dk_weight, eps, interleaved):
    """The struct of a norm + rotation call and its gradient's workspace size, from the tensors' metadata (an
    output that is None is allocated by the caller)."""
    rows, hq, d, qs = _rows_of_heads("q", q)
    _, hkv, d_k, ks = _rows_of_heads("k", k, q)
    if d_k != d or q[0][:-2] != k[0][:-2]:
        raise ValueError(f"q and k must agree on every dimension but the heads, got {tuple(q[0])} and {tuple(k[0])}")
    max_pos, rot = _rotation(q, d, rows, q_weight, k_weight, cos_sin, positions, True)
    _, _, dtype, dev = q
    for name, t, like in (("q_out", q_out, q), ("k_out", k_out, k), ("dq_out", dq_out, q), ("dk_out", dk_out, k)):
        if t is not None:
            _expect(name, t, like[0], dtype, dev)
    strides = []
    for name, t, like in (("dq", dq, q), ("dk", dk, k)):
        if t is not None and t[0] != like[0]:
            raise ValueError(f"{name} must have shape {tuple(like[0])}, got {tuple(t[0])}")
        strides.append(0 if t is None else _rows_of_heads(name, t, q)[3])
    for name, t in (("dq_weight", dq_weight), ("dk_weight", dk_weight)):
        if t is not None:
            _expect(name, t, (d,), _torch()["f32"], dev)
    p = NormRopeProblem(_dtype_code(dtype, "q"), hq, hkv, d, rot, 1 if interleaved else 0, eps, max_pos, rows, qs, ks,
                        *strides)
    return p, int(lib().sdpa_qk_norm_rope_bwd_workspace_size(ctypes.byref(p)))


def sdpa_qk_norm_rope(q, k, q_weight, k_weight, cos_sin=None, positions=None, *, eps=1e-6, interleaved=False, q_out=None,
                      k_out=None, stream=None):
    """Per-head norm of q [..., Hq, D] and k [..., Hkv, D] with the position
    rotation in the same pass (sdpa_qk_norm_rope in include/sdpa.h). Any
    layout's tensors do: the leading dimensions are the tokens. q and k may be
    slices of one projection's output. q_weight, k_weight: [D] of q's dtype.
    cos_sin: float32 [positions, rotary_dim], half cosines and half sines, or
    None for the norm alone; positions: int32, one per token. Returns
    contiguous (q_out, k_out)."""
    if stream is not None:
        return _on(stream, sdpa_qk_norm_rope, locals())
    p, _ = _norm_rope_plan(_meta(q), _meta(k), _meta(q_weight), _meta(k_weight), _meta(cos_sin), _meta(positions),
                           _meta(q_out), _meta(k_out), None, None, None, None, None, None, float(eps), bool(interleaved))
    _refuse_cpu(q)
    like = _torch_state["like"]
    if q_out is None:
        q_out = like(q)
    if k_out is None:
        k_out = like(k)
    _launch("sdpa_qk_norm_rope", q.device, ctypes.byref(p), q.data_ptr(), k.data_ptr(), q_weight.data_ptr(),
            k_weight.data_ptr(), _addr(cos_sin), _addr(positions), q_out.data_ptr(), k_out.data_ptr())
    return q_out, k_out


def sdpa_qk_norm_rope_bwd(dq_out, dk_out, q, k, q_weight, k_weight, cos_sin=None, positions=None, *, eps=1e-6,
                          interleaved=False, dq=None, dk=None, dq_weight=None, dk_weight=None, workspace=None,
                          stream=None):
    """Gradient of sdpa_qk_norm_rope: from the (contiguous) gradients of its
    outputs and its inputs, returns (dq, dk, dq_weight, dk_weight), the weights'
    in float32. dq and dk may be slices of one fused gradient's rows. Bitwise
    reproducible."""
    if stream is not None:
        return _on(stream, sdpa_qk_norm_rope_bwd, locals())
    p, need = _norm_rope_plan(_meta(q), _meta(k), _meta(q_weight), _meta(k_weight), _meta(cos_sin), _meta(positions),
                              None, None, _meta(dq), _meta(dk), _meta(dq_out), _meta(dk_out), _meta(dq_weight),
                              _meta(dk_weight), float(eps), bool(interleaved))
    _refuse_cpu(q)
    dev, f32 = q.device, _torch_state["f32"]
    like = _torch_state["like"]
    dq = like(q) if dq is None else dq
    dk = like(k) if dk is None else dk
    dq_weight = like(q_weight, dtype=f32) if dq_weight is None else dq_weight
    dk_weight = like(q_weight, dtype=f32) if dk_weight is None else dk_weight
    if workspace is None:
        workspace = dq_weight.new_empty(max(need // 4, 4))
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {dev}")
    _launch("sdpa_qk_norm_rope_bwd", dev, ctypes.byref(p), dq_out.data_ptr(), dk_out.data_ptr(), q.data_ptr(),
            k.data_ptr(), q_weight.data_ptr(), k_weight.data_ptr(), _addr(cos_sin), _addr(positions), dq.data_ptr(),
            dk.data_ptr(), dq_weight.data_ptr(), dk_weight.data_ptr(), workspace.data_ptr(), workspace.nbytes)
    return dq, dk, dq_weight, dk_weight


CACHE_LAYOUTS = ("nhd", "hnd")  # [pages, page_size, Hkv, D] and [pages, Hkv, page_size, D]


def _paged_problem(q, hq, k_cache, v_cache, block_table, kv_lens, cu_seqlens_q, cache_layout, total_q, seqlen_q, seqlen_kv,
                   mask_type, window_left, scale, q_stride, k_stride, v_stride) -> PagedProblem:
    """sdpa_paged_problem of a batch over a cache, checked from the tensors'
    metadata. Cache strides are free but for contiguous head_dim, so a cache
    may be a slice of a larger tensor."""
    if cache_layout not in CACHE_LAYOUTS:
        raise ValueError(f"cache_layout must be one of {CACHE_LAYOUTS}, got {cache_layout!r}")
    _, _, dtype, dev = q
    i32 = _torch()["i32"]
    for name, (shape, st, got, got_dev) in (("k_cache", k_cache), ("v_cache", v_cache)):
        if len(shape) != 4 or got is not dtype or got_dev != dev or st[3] != 1:
            raise ValueError(f"{name} must be a 4-dimensional {dtype} tensor on {dev} with contiguous head_dim, got "
                             f"{got} {tuple(shape)} on {got_dev}")
    (ks, k_st), (vs, v_st) = k_cache[:2], v_cache[:2]
    if ks[:3] != vs[:3]:
        raise ValueError(f"k_cache and v_cache must agree on every dimension but the last, got {tuple(ks)} and {tuple(vs)}")
    tab, tab_st, tab_dtype, tab_dev = block_table
    if (len(tab) != 2 or tab_dtype is not i32 or tab_dev != dev or (tab[1] > 1 and tab_st[1] != 1)
            or (tab[0] > 1 and tab_st[0] < tab[1])):  # an expanded row too: a stride of zero stands for contiguous rows
        raise ValueError(f"block_table must be a 2-D int32 [batch, pages] tensor on {dev} with contiguous rows that do "
                         "not overlap")
    batch, max_pages = tab
    _expect("kv_lens", kv_lens, (batch,), i32, dev)
    _expect("cu_seqlens_q", cu_seqlens_q, (batch + 1,), i32, dev)
    slot, head = (1, 2) if cache_layout == "nhd" else (2, 1)
    pages, hkv, d, dv = ks[0], ks[head], ks[3], vs[3]
    # a dimension of one entry may carry any stride: its own row's width stands for it
    return PagedProblem(_dtype_code(dtype, "q"), batch, hq, hkv, d, dv, total_q, seqlen_q,
                        min(max_pages * ks[slot], PAGED_KEYS_MAX) if seqlen_kv is None else seqlen_kv, ks[slot], pages,
                        max_pages, mask_type, window_left, scale, tab_st[0] if batch > 1 else 0,
                        k_st[0] if pages > 1 else d, k_st[slot],
                        k_st[head] if hkv > 1 else d, v_st[0] if pages > 1 else dv, v_st[slot],
                        v_st[head] if hkv > 1 else dv, q_stride, k_stride, v_stride)


@functools.lru_cache(maxsize=_PLANS)
def _append_plan(k, v, k_cache, v_cache, block_table, kv_lens, cu_seqlens_q, cache_layout, q, q_weight, k_weight, cos_sin,
                 positions, q_out, eps, interleaved):
    """The structs of an append (the second None without q)."""
    rows, hkv, d, ks = _rows_of_heads("k", k)
    rows_v, hkv_v, dv, vs = _rows_of_heads("v", v, k)
    if len(k[0]) != 3 or len(v[0]) != 3 or rows != rows_v or hkv != hkv_v:
        raise ValueError(f"k and v must be [tokens, heads, width] of the same tokens and heads, got {tuple(k[0])} and "
                         f"{tuple(v[0])}")
    hq, qs, n = hkv, 0, None
    if q is not None:
        rows_q, hq, d_q, qs = _rows_of_heads("q", q, k)
        if len(q[0]) != 3 or rows_q != rows or d_q != d:
            raise ValueError(f"q must be [tokens, heads, head_dim] of k's tokens and head_dim, got {tuple(q[0])}")
        if q_weight is None or k_weight is None:
            raise ValueError("q needs q_weight and k_weight")
        max_pos, rot = _rotation(q, d, rows, q_weight, k_weight, cos_sin, positions, False)
        n = NormRopeProblem(0, 0, 0, 0, rot, 1 if interleaved else 0, eps, max_pos)
        if q_out is not None:
            _expect("q_out", q_out, q[0], q[2], q[3])
    elif not (q_weight is k_weight is cos_sin is positions is q_out is None):
        raise ValueError("weights, cos_sin, positions and q_out go with q")
    p = _paged_problem(k, hq, k_cache, v_cache, block_table, kv_lens, cu_seqlens_q, cache_layout, rows, 0, 0,
                       MASKS["none"], -1, 0.0, qs, ks, vs)
    if p.num_heads_kv != hkv or p.head_dim != d or p.head_dim_v != dv:
        raise ValueError(f"k and v {tuple(k[0])}, {tuple(v[0])} do not fit the caches {tuple(k_cache[0])}, "
                         f"{tuple(v_cache[0])} in layout {cache_layout}")
    return p, n


@functools.lru_cache(maxsize=_PLANS)
def _paged_plan(q, k_cache, v_cache, block_table, kv_lens, cu_seqlens_q, max_seqlen_q, max_seqlen_kv, cache_layout, mask,
                window_left, window_right, scale, out, lse):
    """The struct of an attention call over a cache, and its workspace size."""
    rows, hq, d, qs = _rows_of_heads("q", q)
    if len(q[0]) != 3:
        raise ValueError(f"q must be [tokens, heads, head_dim], got {tuple(q[0])}")
    if window_right not in (-1, 0):
        raise ValueError(f"a paged window is (left, -1 or 0), got ({window_left}, {window_right})")
    if window_right == 0 and mask == "none":
        raise ValueError("a window that ends at the diagonal goes with mask causal_br")
    for name, n in (("the window", window_left), ("max_seqlen_q", max_seqlen_q), ("max_seqlen_kv", max_seqlen_kv or 0)):
        if not -2 ** 31 <= n < 2 ** 31:  # the struct's field would keep its low bits
            raise ValueError(f"{name} must fit 32 bits, got {n}")
    p = _paged_problem(q, hq, k_cache, v_cache, block_table, kv_lens, cu_seqlens_q, cache_layout, rows, max_seqlen_q,
                       max_seqlen_kv, MASKS[mask], window_left, d ** -0.5 if scale is None else scale, qs, 0, 0)
    if p.head_dim != d or hq % p.num_heads_kv:
        raise ValueError(f"q {tuple(q[0])} does not fit the cache {tuple(k_cache[0])} in layout {cache_layout}")
    if out is not None:
        _expect("out", out, (rows, hq, p.head_dim_v), q[2], q[3])
    if lse is not None:
        _expect("lse", lse, (rows, hq), _torch()["f32"], q[3])
    return p, sdpa_paged_fwd_workspace_size(p)


def sdpa_check_paged(p: PagedProblem) -> int:
    return int(lib().sdpa_check_paged(ctypes.byref(p)))


def sdpa_paged_append(k, v, k_cache, v_cache, block_table, kv_lens, cu_seqlens_q, *, cache_layout="nhd", q=None,
                      q_weight=None, k_weight=None, cos_sin=None, positions=None, eps=1e-6, interleaved=False,
                      q_out=None, stream=None):
    """Write the new tokens' k [T, Hkv, D] and v [T, Hkv, Dv] into their pages
    of k_cache and v_cache (sdpa_paged_append in include/sdpa.h). kv_lens count
    the new tokens already. With q [T, Hq, D] (and q_weight, k_weight), k is
    normed and rotated on its way into the cache and q into q_out, as by
    sdpa_qk_norm_rope; positions default to the cache positions. Returns q_out
    (None without q). k, v and q may be slices of one projection's output."""
    if stream is not None:
        return _on(stream, sdpa_paged_append, locals())
    p, n = _append_plan(_meta(k), _meta(v), _meta(k_cache), _meta(v_cache), _meta(block_table), _meta(kv_lens),
                        _meta(cu_seqlens_q), cache_layout, _meta(q), _meta(q_weight), _meta(k_weight), _meta(cos_sin),
                        _meta(positions), _meta(q_out), float(eps), bool(interleaved))
    _refuse_cpu(k)
    if q is not None and q_out is None:
        q_out = _torch_state["like"](q)
    _launch("sdpa_paged_append", k.device, ctypes.byref(p), None if n is None else ctypes.byref(n), _addr(q),
            k.data_ptr(), v.data_ptr(), _addr(q_weight), _addr(k_weight), _addr(cos_sin), _addr(positions), _addr(q_out),
            k_cache.data_ptr(), v_cache.data_ptr(), cu_seqlens_q.data_ptr(), kv_lens.data_ptr(), block_table.data_ptr())
    return q_out


def sdpa_paged_fwd_workspace_size(p: PagedProblem) -> int:
    return int(lib().sdpa_paged_fwd_workspace_size(ctypes.byref(p)))


def sdpa_paged_fwd(q, k_cache, v_cache, block_table, kv_lens, cu_seqlens_q, *, max_seqlen_q, max_seqlen_kv=None,
                   cache_layout="nhd", mask="causal_br", window=(-1, -1), scale=None, out=None, lse=None, workspace=None,
                   stream=None):
    """Attention of the new tokens q [T, Hq, D] over a paged cache that holds
    their keys and values already (sdpa_paged_fwd in include/sdpa.h).
    k_cache, v_cache: [pages, page_size, Hkv, D] ("nhd") or [pages, Hkv,
    page_size, D] ("hnd"); block_table int32 [batch, pages per sequence];
    kv_lens int32 [batch], the new tokens included; cu_seqlens_q int32
    [batch + 1]. max_seqlen_q, max_seqlen_kv: the most new tokens and the
    longest kv_len (default: what the block table can hold). mask: "causal_br"
    or "none"; window = (left, -1 or 0), with "none" (-1, -1). q may be a slice
    of wider rows whose spacing is a multiple of D elements. Returns (o [T, Hq,
    Dv], lse float32 [T, Hq]); rows behind the last sequence are left as they
    are. A workspace of PAGED_WORKSPACE_MAX bytes serves every shape."""
    if stream is not None:
        return _on(stream, sdpa_paged_fwd, locals())
    p, need = _paged_plan(_meta(q), _meta(k_cache), _meta(v_cache), _meta(block_table), _meta(kv_lens),
                          _meta(cu_seqlens_q), int(max_seqlen_q), None if max_seqlen_kv is None else int(max_seqlen_kv),
                          cache_layout, mask, int(window[0]), int(window[1]), None if scale is None else float(scale),
                          _meta(out), _meta(lse))
    _refuse_cpu(q)
    dev = q.device
    if out is None:
        out = q.new_empty((p.total_q, p.num_heads_q, p.head_dim_v))
    if lse is None:
        lse = q.new_empty((p.total_q, p.num_heads_q), dtype=_torch_state["f32"])
    if workspace is None:
        workspace = lse.new_empty(max(need // 4, 64))
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {dev}")
    _launch("sdpa_paged_fwd", dev, ctypes.byref(p), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
            out.data_ptr(), lse.data_ptr(), cu_seqlens_q.data_ptr(), kv_lens.data_ptr(), block_table.data_ptr(),
            workspace.data_ptr(), workspace.nbytes)
    return out, lse


def sdpa_selftest_bounded_wait(limit_us: int = 20000, stream=None) -> None:
    """Launch the bounded-wait self-test (records SDPA_ERR_TIMEOUT on the device)."""
    rc = lib().sdpa_selftest_bounded_wait(int(limit_us), _stream(stream))
    if rc:
        raise SdpaError(rc, "sdpa_selftest_bounded_wait")
