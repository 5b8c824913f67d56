"""Thin ctypes binding of libsage.so (the C ABI declared in include/sage.h).

Argument marshalling only: every step of the quantized attention runs in the
library's CUDA kernels.  torch supplies device memory and the current stream.
There is no fallback: if the library is missing or cannot load, importing
this module raises.
"""
from __future__ import annotations

import ctypes
import os

from . import _build

F16, BF16, Q8, Q4 = 0, 1, 2, 3
HND, NHD = 0, 1
OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_CUDA, ERR_DEVICE_TIMEOUT = range(6)
STATUS_NAMES = ["OK", "INVALID_ARG", "UNSUPPORTED", "WORKSPACE", "CUDA", "DEVICE_TIMEOUT"]

# Every entry point declared in include/sage.h.
EXPORTS = (
    "sage_workspace_bytes", "sage_workspace_bytes_varlen", "sage_quant_prologue",
    "sage_quant_prologue_varlen", "sage_attn_quantized", "sage_attn_fwd",
    "sage_attn_fwd_varlen", "sage_debug_qk_int32", "sage_debug_e4m3",
    "sage_debug_set_fault", "sage_debug_set_prologue_launches", "sage_device_status",
    "sage_last_error",
    "sage_kv_stats_noalloc", "sage_launch_count", "sage_quant_prologue_strided",
    "sage_attn_fwd_strided", "sage_quant_prologue_pv16", "sage_attn_fwd_pv16",
    "sage_workspace_bytes_host", "sage_attn_fwd_host", "sage_attn_fwd_host_pv16",
    "sage_debug_pv_accum", "sage_debug_set_fault_launches", "sage_kv_stats_noalloc_status",
    "sage_debug_tc_rate", "sage_workspace_bytes_varlen_host", "sage_attn_fwd_varlen_host",
    "sage_debug_set_host_fail_chunk",
    "sage_rope", "sage_workspace_bytes_paged", "sage_kv_append", "sage_attn_paged",
    "sage_rope_axes", "sage_kv_append_axes", "sage_kv_gather", "sage_paged_step",
    "sage_paged_trim",
)


class SageError(RuntimeError):
    def __init__(self, status: int, where: str, reason: str):
        name = STATUS_NAMES[status] if 0 <= status < len(STATUS_NAMES) else str(status)
        super().__init__(f"{where}: SAGE_ERR_{name}: {reason}")
        self.status = status


class Quantized(ctypes.Structure):
    """Mirror of sage_quantized (pointers into the workspace)."""
    _fields_ = [
        ("nseg", ctypes.c_int64), ("Hq", ctypes.c_int64), ("Hkv", ctypes.c_int64),
        ("Lq", ctypes.c_int64), ("Lk", ctypes.c_int64), ("D", ctypes.c_int64),
        ("Dp", ctypes.c_int64), ("dtype", ctypes.c_int32), ("varlen", ctypes.c_int32),
        ("total_q", ctypes.c_int64), ("total_k", ctypes.c_int64),
        ("max_q", ctypes.c_int32), ("max_k", ctypes.c_int32),
        ("q_head_rows", ctypes.c_int64), ("k_head_rows", ctypes.c_int64),
        ("q_rows", ctypes.c_int64), ("k_rows", ctypes.c_int64),
        ("v_rows", ctypes.c_int64), ("v_cols", ctypes.c_int64),
        ("cu_q", ctypes.c_void_p), ("cu_k", ctypes.c_void_p),
        ("q16", ctypes.c_void_p), ("k16", ctypes.c_void_p), ("v8", ctypes.c_void_p),
        ("s_q", ctypes.c_void_p), ("s_k", ctypes.c_void_p), ("s_v", ctypes.c_void_p),
        ("k_mean", ctypes.c_void_p), ("stats", ctypes.c_void_p),
        ("status", ctypes.c_void_p), ("v_fp16", ctypes.c_int32),
    ]


class _CacheC(ctypes.Structure):
    """Mirror of sage_paged_cache."""
    _fields_ = [
        ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
        ("k_mean", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
        ("num_pages", ctypes.c_int64), ("page_size", ctypes.c_int64), ("Hkv", ctypes.c_int64),
        ("D", ctypes.c_int64), ("page_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64),
        ("head_stride", ctypes.c_int64), ("kind", ctypes.c_int32),
        ("k_groups", ctypes.c_void_p), ("v_groups", ctypes.c_void_p),
    ]


class _BatchC(ctypes.Structure):
    """Mirror of sage_paged_batch."""
    _fields_ = [
        ("cu_q", ctypes.c_void_p), ("kv_lens", ctypes.c_void_p), ("block_table", ctypes.c_void_p),
        ("nseq", ctypes.c_int64), ("total_q", ctypes.c_int64), ("table_stride", ctypes.c_int64),
        ("table_width", ctypes.c_int64), ("max_q", ctypes.c_int32), ("max_kv", ctypes.c_int32),
    ]


class _PoolC(ctypes.Structure):
    """Mirror of sage_page_pool."""
    _fields_ = [
        ("free_pages", ctypes.c_void_p), ("left", ctypes.c_void_p), ("table", ctypes.c_void_p),
        ("lens", ctypes.c_void_p), ("marks", ctypes.c_void_p), ("num_pages", ctypes.c_int64),
        ("page_size", ctypes.c_int64), ("max_requests", ctypes.c_int64),
        ("table_stride", ctypes.c_int64), ("table_width", ctypes.c_int64),
    ]


class _PlanC(ctypes.Structure):
    """Mirror of sage_paged_plan."""
    _fields_ = [
        ("cu_q", ctypes.c_void_p), ("kv_lens", ctypes.c_void_p), ("block_table", ctypes.c_void_p),
        ("positions", ctypes.c_void_p), ("slots", ctypes.c_void_p), ("denied", ctypes.c_void_p),
        ("n", ctypes.c_int64), ("rows", ctypes.c_int64), ("table_stride", ctypes.c_int64),
        ("table_width", ctypes.c_int64), ("max_q", ctypes.c_int32), ("max_kv", ctypes.c_int32),
    ]


def _load():
    path = _build.LIB
    if not _build.up_to_date():
        path = _build.build()
    lib = ctypes.CDLL(path)
    P, I64, I, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
    F = ctypes.c_float
    QP = ctypes.POINTER(Quantized)
    sig = {
        "sage_workspace_bytes": ([I64] * 6, SZ),
        "sage_workspace_bytes_host": ([I64] * 7, SZ),
        "sage_attn_fwd_host": ([P, P, P, P, I64, I64, I64, I64, I64, I64, I, I, F, I, I64, P, SZ,
                                P], I),
        "sage_attn_fwd_host_pv16": ([P, P, P, P, I64, I64, I64, I64, I64, I64, I, I, F, I, I64, P,
                                     SZ, P], I),
        "sage_workspace_bytes_varlen": ([I64] * 6, SZ),
        "sage_workspace_bytes_varlen_host": ([I64] * 7, SZ),
        "sage_attn_fwd_varlen_host": ([P, P, P, P, P, P, I64, I64, I64, I, I, I64, I64, I64, I,
                                       F, I, I64, P, SZ, P], I),
        "sage_quant_prologue": ([P, P, P, I, I, I64, I64, I64, I64, I64, I64, P, SZ, QP, P], I),
        "sage_quant_prologue_varlen": ([P, P, P, I, P, P, I64, I64, I64, I, I, I64, I64, I64,
                                        P, SZ, QP, P], I),
        "sage_quant_prologue_strided": ([P, P, P, I, I64, I64, I64, I64, I64, I64, P, P, P, SZ,
                                         QP, P], I),
        "sage_attn_fwd_strided": ([P, P, P, P, I64, I64, I64, I64, I64, I64, P, P, I, I, F, I,
                                   P, SZ, P], I),
        "sage_quant_prologue_pv16": ([P, P, P, I, I, I64, I64, I64, I64, I64, I64, P, SZ, QP,
                                      P], I),
        "sage_attn_fwd_pv16": ([P, P, P, P, I64, I64, I64, I64, I64, I64, I, I, F, I, P, SZ, P],
                               I),
        "sage_attn_quantized": ([QP, P, I, I, F, P], I),
        "sage_attn_fwd": ([P, P, P, P, I64, I64, I64, I64, I64, I64, I, I, F, I, P, SZ, P], I),
        "sage_attn_fwd_varlen": ([P, P, P, P, P, P, I64, I64, I64, I, I, I64, I64, I64, I, F,
                                  I, P, SZ, P], I),
        "sage_debug_qk_int32": ([QP, I64, I64, I64, I64, P, P], I),
        "sage_debug_e4m3": ([P, P, I64, P], I),
        "sage_debug_pv_accum": ([P, P, I64, I64, P, P, P], I),
        "sage_debug_set_fault": ([I, ctypes.c_uint64], None),
        "sage_debug_set_prologue_launches": ([I], None),
        "sage_debug_set_fault_launches": ([I], None),
        "sage_debug_set_host_fail_chunk": ([I], None),
        "sage_debug_tc_rate": ([I, I64, P, P], I),
        "sage_kv_stats_noalloc_status": ([P], I),
        "sage_device_status": ([P, P], I),
        "sage_last_error": ([], ctypes.c_char_p),
        "sage_kv_stats_noalloc": ([P, P, I, I, I64, I64, I64, I64, P, P, P], I),
        "sage_launch_count": ([], ctypes.c_uint64),
        "sage_rope": ([P, P, P, P, I, I64, I64, I64, I64, P, P, P, P, P, I, P, I64, I, F, I, P], I),
        "sage_workspace_bytes_paged": ([], SZ),
        "sage_kv_append": ([P, P, P, P, P, P, I, I64, P, P, P, P, P, I64, I, F, P, SZ, P], I),
        "sage_attn_paged": ([P, P, P, P, P, I, I64, P, I64, I64, F, P, SZ, P], I),
        "sage_rope_axes": ([P, P, P, P, I, I64, I64, I64, I64, P, P, P, P, P, I, I64, I64, P, P,
                            I64, I, F, I, P], I),
        "sage_kv_append_axes": ([P, P, P, P, P, P, I, I64, P, P, P, P, P, I, I64, I64, P, P, I64,
                                 I, F, P, SZ, P], I),
        "sage_kv_gather": ([P, P, P, P, I, P, P, P, SZ, P], I),
        "sage_paged_step": ([P, P, P, P, P, SZ, P], I),
        "sage_paged_trim": ([P, P, P, I64, P, SZ, P], I),
    }
    for name, (args, res) in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    return lib


_lib = _load()
lib = _lib


def last_error() -> str:
    return _lib.sage_last_error().decode()


def launch_count() -> int:
    """Kernels this library has launched in this process (host-side count)."""
    return int(_lib.sage_launch_count())


def _check(rc: int, where: str):
    if rc != OK:
        raise SageError(rc, where, last_error())


def _stream(stream):
    if stream is None:
        import torch
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return ctypes.c_void_p(stream)
    return ctypes.c_void_p(stream.cuda_stream)


def _ptr(t):
    return ctypes.c_void_p(0 if t is None else t.data_ptr())


def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.float16:
        return F16
    if t.dtype == torch.bfloat16:
        return BF16
    raise TypeError(f"q/k/v must be float16 or bfloat16, got {t.dtype}")


def _require_dense(where, q, k, v, out=None):
    """The dense and packed entry points read q, k, v (and write out) as
    contiguous arrays of one dtype on a CUDA device.  Anything else is
    refused here, before any call: a view must go through the *_strided
    calls, which take its strides."""
    for name, t in (("q", q), ("k", k), ("v", v)):
        if not t.is_cuda:
            raise ValueError(f"{where}: {name} is not on a CUDA device")
        if not t.is_contiguous():
            raise ValueError(f"{where}: {name} is not contiguous; pass views to "
                             f"quant_prologue_strided / attn_fwd_strided")
        if t.dtype != q.dtype:
            raise TypeError(f"{where}: {name} is {t.dtype}, q is {q.dtype}")
    if out is not None:
        import torch
        if not out.is_cuda or not out.is_contiguous() or out.dtype != torch.float32:
            raise ValueError(f"{where}: out must be a contiguous float32 CUDA tensor")
        if tuple(out.shape) != tuple(q.shape):
            raise ValueError(f"{where}: out has shape {tuple(out.shape)}, q {tuple(q.shape)}")


def _layout_code(layout) -> int:
    if layout in (HND, "HND"):
        return HND
    if layout in (NHD, "NHD"):
        return NHD
    raise ValueError(f"layout must be 'HND' or 'NHD', got {layout!r}")


def _dims(q, k, layout):
    if layout == HND:
        B, Hq, Lq, D = q.shape
        _, Hkv, Lk, _ = k.shape
    else:
        B, Lq, Hq, D = q.shape
        _, Lk, Hkv, _ = k.shape
    return B, Hq, Hkv, Lq, Lk, D


def workspace_bytes(B, Hq, Hkv, Lq, Lk, D) -> int:
    return int(_lib.sage_workspace_bytes(B, Hq, Hkv, Lq, Lk, D))


def workspace_bytes_varlen(nseq, total_q, total_k, Hq, Hkv, D) -> int:
    return int(_lib.sage_workspace_bytes_varlen(nseq, total_q, total_k, Hq, Hkv, D))


def alloc_workspace(nbytes: int, device="cuda"):
    import torch
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


def quant_prologue(q, k, v, layout="HND", ws=None, stream=None) -> Quantized:
    _require_dense("quant_prologue", q, k, v)
    lay = _layout_code(layout)
    B, Hq, Hkv, Lq, Lk, D = _dims(q, k, lay)
    if ws is None:
        ws = alloc_workspace(workspace_bytes(B, Hq, Hkv, Lq, Lk, D), q.device)
    qt = Quantized()
    rc = _lib.sage_quant_prologue(_ptr(q), _ptr(k), _ptr(v), _dtype_code(q), lay, B, Hq,
                                  Hkv, Lq, Lk, D, _ptr(ws), ws.numel(), ctypes.byref(qt),
                                  _stream(stream))
    _check(rc, "sage_quant_prologue")
    qt._ws = ws
    return qt


def quant_prologue_pv16(q, k, v, layout="HND", ws=None, stream=None) -> Quantized:
    """Prologue of the FP16-PV variant: INT8 Q/K as usual, V kept in fp16."""
    _require_dense("quant_prologue_pv16", q, k, v)
    lay = _layout_code(layout)
    B, Hq, Hkv, Lq, Lk, D = _dims(q, k, lay)
    if ws is None:
        ws = alloc_workspace(workspace_bytes(B, Hq, Hkv, Lq, Lk, D), q.device)
    qt = Quantized()
    rc = _lib.sage_quant_prologue_pv16(_ptr(q), _ptr(k), _ptr(v), _dtype_code(q), lay, B, Hq,
                                       Hkv, Lq, Lk, D, _ptr(ws), ws.numel(), ctypes.byref(qt),
                                       _stream(stream))
    _check(rc, "sage_quant_prologue_pv16")
    qt._ws = ws
    return qt


def quant_prologue_varlen(q, k, v, cu_q, cu_k, max_q, max_k, ws=None, stream=None):
    _require_dense("quant_prologue_varlen", q, k, v)
    total_q, Hq, D = q.shape
    total_k, Hkv, _ = k.shape
    nseq = cu_q.numel() - 1
    if ws is None:
        ws = alloc_workspace(workspace_bytes_varlen(nseq, total_q, total_k, Hq, Hkv, D),
                             q.device)
    qt = Quantized()
    rc = _lib.sage_quant_prologue_varlen(_ptr(q), _ptr(k), _ptr(v), _dtype_code(q),
                                         _ptr(cu_q), _ptr(cu_k), nseq, total_q, total_k,
                                         int(max_q), int(max_k), Hq, Hkv, D, _ptr(ws),
                                         ws.numel(), ctypes.byref(qt), _stream(stream))
    _check(rc, "sage_quant_prologue_varlen")
    qt._ws = ws
    return qt


def attn_quantized(qt: Quantized, out, layout="HND", is_causal=False, sm_scale=None,
                   stream=None):
    rc = _lib.sage_attn_quantized(ctypes.byref(qt), _ptr(out), _layout_code(layout),
                                  int(bool(is_causal)), float(sm_scale or 0.0),
                                  _stream(stream))
    _check(rc, "sage_attn_quantized")
    return out


def attn_fwd(q, k, v, out, layout="HND", is_causal=False, sm_scale=None, ws=None,
             stream=None):
    _require_dense("attn_fwd", q, k, v, out)
    lay = _layout_code(layout)
    B, Hq, Hkv, Lq, Lk, D = _dims(q, k, lay)
    if ws is None:
        ws = alloc_workspace(workspace_bytes(B, Hq, Hkv, Lq, Lk, D), q.device)
    rc = _lib.sage_attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(out), B, Hq, Hkv, Lq, Lk, D,
                            lay, int(bool(is_causal)), float(sm_scale or 0.0),
                            _dtype_code(q), _ptr(ws), ws.numel(), _stream(stream))
    _check(rc, "sage_attn_fwd")
    return out


def attn_fwd_pv16(q, k, v, out, layout="HND", is_causal=False, sm_scale=None, ws=None,
                 stream=None):
    """Prologue + FP16-PV attention (dense)."""
    _require_dense("attn_fwd_pv16", q, k, v, out)
    lay = _layout_code(layout)
    B, Hq, Hkv, Lq, Lk, D = _dims(q, k, lay)
    if ws is None:
        ws = alloc_workspace(workspace_bytes(B, Hq, Hkv, Lq, Lk, D), q.device)
    rc = _lib.sage_attn_fwd_pv16(_ptr(q), _ptr(k), _ptr(v), _ptr(out), B, Hq, Hkv, Lq, Lk, D,
                                 lay, int(bool(is_causal)), float(sm_scale or 0.0),
                                 _dtype_code(q), _ptr(ws), ws.numel(), _stream(stream))
    _check(rc, "sage_attn_fwd_pv16")
    return out


def workspace_bytes_host(B, Hq, Hkv, Lq, Lk, D, chunk_kv_heads=0) -> int:
    return int(_lib.sage_workspace_bytes_host(B, Hq, Hkv, Lq, Lk, D, int(chunk_kv_heads)))


def attn_fwd_host(q, k, v, out, layout="HND", is_causal=False, sm_scale=None,
                  chunk_kv_heads=0, ws=None, stream=None, pv16=False):
    """Attention on host tensors (page-locked for overlap): the library copies
    chunks in, computes them and copies the output back, pipelined.  `out`
    is a host float32 tensor of q's shape; `stream` completes when it is
    filled."""
    import torch
    for name, t in (("q", q), ("k", k), ("v", v), ("out", out)):
        if t.is_cuda or not t.is_contiguous():
            raise ValueError(f"attn_fwd_host: {name} must be a contiguous host tensor")
    if k.dtype != q.dtype or v.dtype != q.dtype:
        raise TypeError("attn_fwd_host: q, k and v must share one dtype")
    if out.dtype != torch.float32 or tuple(out.shape) != tuple(q.shape):
        raise ValueError("attn_fwd_host: out must be float32 with q's shape")
    lay = _layout_code(layout)
    B, Hq, Hkv, Lq, Lk, D = _dims(q, k, lay)
    if ws is None:
        ws = alloc_workspace(workspace_bytes_host(B, Hq, Hkv, Lq, Lk, D, chunk_kv_heads))
    fn = _lib.sage_attn_fwd_host_pv16 if pv16 else _lib.sage_attn_fwd_host
    rc = fn(_ptr(q), _ptr(k), _ptr(v), _ptr(out), B, Hq, Hkv, Lq, Lk, D, lay,
            int(bool(is_causal)), float(sm_scale or 0.0), _dtype_code(q), int(chunk_kv_heads),
            _ptr(ws), ws.numel(), _stream(stream))
    _check(rc, "sage_attn_fwd_host_pv16" if pv16 else "sage_attn_fwd_host")
    return out


def attn_fwd_varlen(q, k, v, out, cu_q, cu_k, max_q, max_k, is_causal=False,
                    sm_scale=None, ws=None, stream=None):
    _require_dense("attn_fwd_varlen", q, k, v, out)
    total_q, Hq, D = q.shape
    total_k, Hkv, _ = k.shape
    nseq = cu_q.numel() - 1
    if ws is None:
        ws = alloc_workspace(workspace_bytes_varlen(nseq, total_q, total_k, Hq, Hkv, D),
                             q.device)
    rc = _lib.sage_attn_fwd_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(cu_q),
                                   _ptr(cu_k), nseq, total_q, total_k, int(max_q),
                                   int(max_k), Hq, Hkv, D, int(bool(is_causal)),
                                   float(sm_scale or 0.0), _dtype_code(q), _ptr(ws),
                                   ws.numel(), _stream(stream))
    _check(rc, "sage_attn_fwd_varlen")
    return out


def view_strides(t, layout) -> tuple:
    """(batch, head, token) strides in elements of a q/k/v view in `layout`;
    the channel stride must be 1."""
    lay = _layout_code(layout)
    st = t.stride()
    if st[3] != 1:
        raise ValueError(f"strided views need contiguous channels (channel stride {st[3]})")
    return (st[0], st[1], st[2]) if lay == HND else (st[0], st[2], st[1])


def _strides_arg(vals):
    return (ctypes.c_int64 * 3)(*[int(x) for x in vals])


def _kv_strides(k, v, layout):
    ks, vs = view_strides(k, layout), view_strides(v, layout)
    if ks != vs:
        raise ValueError(f"k and v views must share their strides (k {ks}, v {vs})")
    return ks


def quant_prologue_strided(q, k, v, layout="HND", ws=None, stream=None) -> Quantized:
    """Prologue on q/k/v views (e.g. slices of one fused projection)."""
    lay = _layout_code(layout)
    B, Hq, Hkv, Lq, Lk, D = _dims(q, k, lay)
    if ws is None:
        ws = alloc_workspace(workspace_bytes(B, Hq, Hkv, Lq, Lk, D), q.device)
    qt = Quantized()
    rc = _lib.sage_quant_prologue_strided(
        _ptr(q), _ptr(k), _ptr(v), _dtype_code(q), B, Hq, Hkv, Lq, Lk, D,
        _strides_arg(view_strides(q, lay)), _strides_arg(_kv_strides(k, v, lay)), _ptr(ws),
        ws.numel(), ctypes.byref(qt), _stream(stream))
    _check(rc, "sage_quant_prologue_strided")
    qt._ws = ws
    return qt


def attn_fwd_strided(q, k, v, out, layout="HND", is_causal=False, sm_scale=None, ws=None,
                     stream=None):
    """Prologue + attention on q/k/v views; out is dense fp32 in `layout`."""
    lay = _layout_code(layout)
    B, Hq, Hkv, Lq, Lk, D = _dims(q, k, lay)
    if ws is None:
        ws = alloc_workspace(workspace_bytes(B, Hq, Hkv, Lq, Lk, D), q.device)
    rc = _lib.sage_attn_fwd_strided(
        _ptr(q), _ptr(k), _ptr(v), _ptr(out), B, Hq, Hkv, Lq, Lk, D,
        _strides_arg(view_strides(q, lay)), _strides_arg(_kv_strides(k, v, lay)), lay,
        int(bool(is_causal)), float(sm_scale or 0.0), _dtype_code(q), _ptr(ws), ws.numel(),
        _stream(stream))
    _check(rc, "sage_attn_fwd_strided")
    return out


def sageattn(q, k, v, tensor_layout="HND", is_causal=False, sm_scale=None):
    """Drop-in style call: fp16/bf16 q, k, v on the GPU -> fp32 output.  Views
    (for instance the slices of a fused qkv projection) go through the
    strided entry point; a view it cannot serve raises with the reason."""
    import torch
    out = torch.empty(q.shape, dtype=torch.float32, device=q.device)
    if q.is_contiguous() and k.is_contiguous() and v.is_contiguous():
        return attn_fwd(q, k, v, out, tensor_layout, is_causal, sm_scale)
    return attn_fwd_strided(q, k, v, out, tensor_layout, is_causal, sm_scale)


def sageattn_qk_int8_pv_fp16(q, k, v, tensor_layout="HND", is_causal=False, sm_scale=None):
    """The more accurate variant: INT8 QK^T, fp16 P and V (dense inputs)."""
    import torch
    out = torch.empty(q.shape, dtype=torch.float32, device=q.device)
    return attn_fwd_pv16(q, k, v, out, tensor_layout, is_causal, sm_scale)


# ------------------------------------------------------------------ serving
def rope_freqs(rotary_dim, base=10000.0, scaling=None, factor=1.0, original_len=4096, low=1.0,
               high=32.0, device="cuda"):
    """(inv_freq, mscale) for `rope` and `kv_append`: inv_freq float64
    [rotary_dim / 2] on `device`, base ** (-2 i / rotary_dim), scaled for
    lengths beyond `original_len`:
      None        unscaled
      "linear"    every frequency divided by `factor` (positions interpolated)
      "ntk"       base times factor ** (R / (R - 2)): the longest wavelength is
                  stretched by `factor`, the shortest kept
      "by_parts"  frequencies that turn fewer than `low` times in original_len
                  divided by `factor`, those above `high` kept, a linear ramp
                  in the number of turns between
      "yarn"      between the same two ends, rounded outwards to whole pairs, a
                  ramp linear in the pair's index i instead, as models trained
                  with YaRN have it; and mscale = 0.1 ln(factor) + 1"""
    import math
    import torch
    r = int(rotary_dim)
    if r < 2 or r % 2:
        raise ValueError(f"rope_freqs: rotary_dim must be even and positive, got {rotary_dim}")
    if not factor >= 1.0:
        raise ValueError(f"rope_freqs: factor must be at least 1, got {factor}")
    if scaling == "ntk":
        if r == 2:
            raise ValueError("rope_freqs: ntk scaling needs rotary_dim > 2")
        base = base * factor ** (r / (r - 2))
    f = float(base) ** (-torch.arange(r // 2, dtype=torch.float64) * 2 / r)
    mscale = 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling == "by_parts":
        keep = ((original_len * f / (2 * math.pi) - low) / (high - low)).clamp(0, 1)
        f = f * (keep + (1 - keep) / factor)
    elif scaling == "yarn":
        if not (0 < low <= high and base > 1 and original_len > 0):
            raise ValueError("rope_freqs: yarn scaling needs 0 < low <= high, base > 1 and a "
                             "positive original_len")
        # base ** (-2 i / r) * original_len / (2 pi) = n turns, solved for i
        def pair(n):
            return r / 2 * math.log(original_len / (2 * math.pi * n)) / math.log(base)
        first, last = max(math.floor(pair(high)), 0), min(math.ceil(pair(low)), r - 1)
        away = ((torch.arange(r // 2, dtype=torch.float64) - first) /
                max(last - first, 1e-3)).clamp(0, 1)
        f = f * (1 - away + away / factor)
        mscale = 0.1 * math.log(factor) + 1.0
    elif scaling not in (None, "ntk"):
        raise ValueError(f"rope_freqs: unknown scaling {scaling!r}")
    return f.to(device), mscale


# The serving calls run in a few microseconds on the GPU, so their wrappers do:
# plain integers for pointers, one look at the current device, and no torch call
# that a tensor's own methods can answer.
_torch = _get_device = _get_stream = _empty_like = None


def _bind_torch():
    global _torch, _get_device, _get_stream, _empty_like
    import torch
    _empty_like = torch.empty_like
    _get_device, _get_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
    _CODES.update({torch.float16: F16, torch.bfloat16: BF16})
    _torch = torch                # last: other threads take it for a sign that all are set


def _device(where, name, t):
    """(index of the current device, its current stream's handle); t, the
    call's first tensor, is on a CUDA device."""
    if not t.is_cuda:
        _off_device(where, name, t, None)
    if _torch is None:
        _bind_torch()
    d = _get_device()
    return d, _get_stream(d)


def _off_device(where, name, t, dev):
    if not t.is_cuda:
        raise ValueError(f"{where}: {name} is not on a CUDA device")
    raise ValueError(f"{where}: {name} is on {t.device}, the current device is cuda:{dev}")


def _rows3(where, name, t, dev):
    """A (T, H, D) view the serving calls read or write: on the current CUDA
    device, channel stride 1.  Returns its shape and the {token, head} strides
    to pass (None: dense)."""
    shape = t.shape
    if t.get_device() != dev:
        _off_device(where, name, t, dev)
    if t.is_contiguous() and len(shape) == 3:
        return shape, None
    if len(shape) != 3 or t.stride(2) != 1 and shape[2] > 1:
        raise ValueError(f"{where}: {name} must be (T, H, D) with contiguous channels, got shape "
                         f"{tuple(shape)}, strides {t.stride()}")
    return shape, _Strides(t.stride(0), t.stride(1))


def _on_device(where, name, t, dev=None):
    dev = _device(where, name, t)[0] if dev is None else dev
    if t.get_device() != dev:
        _off_device(where, name, t, dev)


def _code16(where, name, t):
    """SAGE_F16 or SAGE_BF16."""
    code = _CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"{where}: {name} must be float16 or bfloat16, got {t.dtype}")
    return code


_CODES: dict = {}
_Strides = ctypes.c_int64 * 2


def _handle(stream, current):
    if stream is None:
        return current
    return stream if isinstance(stream, int) else stream.cuda_stream


def _empty_on(stream, make):
    """Allocates under `stream`, so that the memory is not reused while that
    stream still works on it."""
    if stream is None:
        return make()
    import torch
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream)
    with torch.cuda.stream(stream):
        return make()


def _freqs(where, inv_freq, dev):
    if inv_freq.dtype != _torch.float64 or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
        raise ValueError(f"{where}: inv_freq must be a contiguous 1-D float64 tensor")
    if inv_freq.get_device() != dev:
        _off_device(where, "inv_freq", inv_freq, dev)


def _result(where, name, out, t, stream, dev, dense):
    """`out`, checked, or a new dense tensor of t's shape; with its strides.
    dense: t is dense itself."""
    if out is None:
        if stream is not None:
            return _empty_on(stream, lambda: t.new_empty(t.shape)), None
        return _empty_like(t) if dense else t.new_empty(t.shape), None
    shape, st = _rows3(where, name, out, dev)
    if shape != t.shape:
        raise ValueError(f"{where}: {name} has shape {tuple(shape)}, not {tuple(t.shape)}")
    if out.dtype != t.dtype:
        raise TypeError(f"{where}: {name} is {out.dtype}, not {t.dtype}")
    return out, st


def rope_axes(sections, in_turn=False, device="cuda"):
    """The axis that each channel pair follows, for `rope` and `kv_append`: uint8
    [sum(sections)] on `device`, sections[a] pairs of axis a: one section after
    the other, or with `in_turn` axis 0, 1, 2, 0, 1, 2, ... while an axis has pairs
    left.  Frequencies go by the pair (`rope_freqs`), or by the axis if the
    caller puts those of each axis where its pairs are."""
    import torch
    sections = [int(x) for x in sections]
    if not 1 <= len(sections) <= 8 or min(sections) < 0 or not 1 <= sum(sections) <= 64:
        raise ValueError(f"rope_axes: 1 to 8 sections of 1 to 64 pairs in all, got {sections}")
    order = [a for a, x in enumerate(sections) for _ in range(x)]
    if in_turn:
        nth = [i for x in sections for i in range(x)]
        order = [a for _, a in sorted(zip(nth, order))]
    return torch.tensor(order, dtype=torch.uint8, device=device)


def _axes(where, positions, axes, T, R, dev):
    """Checks positions (A, T) and axes; the arguments that the library takes."""
    shape = positions.shape
    bits = 64 if positions.dtype == _torch.int64 else 32
    if bits == 32 and positions.dtype != _torch.int32 or not 1 <= len(shape) <= 2 or \
            shape[-1] != T or len(shape) == 2 and not 1 <= shape[0] <= 8 or \
            T > 1 and positions.stride(-1) != 1:
        raise ValueError(f"{where}: positions must be int64 or int32, (axes, {T}) with contiguous "
                         f"rows and 1 to 8 axes, got {positions.dtype} {tuple(shape)}")
    if positions.get_device() != dev:
        _off_device(where, "positions", positions, dev)
    ap = 0
    if axes is not None:
        if axes.dtype != _torch.uint8 or axes.shape != (R // 2,) or not axes.is_contiguous():
            raise ValueError(f"{where}: axes must be a contiguous uint8 tensor of {R // 2} entries")
        if axes.get_device() != dev:
            _off_device(where, "axes", axes, dev)
        ap = axes.data_ptr()
    if len(shape) == 1:
        return positions.data_ptr(), bits, 1, T, ap
    return positions.data_ptr(), bits, shape[0], positions.stride(0) if shape[0] > 1 else T, ap


def rope(q, k, positions, inv_freq, interleaved=False, mscale=1.0, inverse=False, q_out=None,
         k_out=None, stream=None, axes=None):
    """Rotary positions of q (T, Hq, D) and k (T, Hkv, D), fp16/bf16 views with
    contiguous channels; k may be None.  positions: int64 or int32 (T,);
    inv_freq: float64 (R/2,), R <= D (see rope_freqs).  Pairs are (i, i + R/2),
    or (2i, 2i + 1) with `interleaved`.  q_out=q (k_out=k) turns in place.
    `inverse` turns back; applied to the outputs' gradients with the same
    mscale it gives the inputs' gradients.  With `axes` (uint8 (R/2,), see
    rope_axes) positions are (A, T), a row for each of up to 8 axes (one row for
    all: positions.expand(A, T)), and pair i turns by its axis' position.  Returns
    (q_out, k_out)."""
    dev, current = _device("rope", "q", q)
    (T, Hq, D), qs = _rows3("rope", "q", q, dev)
    dtype = _code16("rope", "q", q)
    many = None
    bits = 64 if positions.dtype == _torch.int64 else 32
    if axes is not None:
        _freqs("rope", inv_freq, dev)
        many = _axes("rope", positions, axes, T, 2 * inv_freq.shape[0], dev)
    elif bits == 32 and positions.dtype != _torch.int32 or positions.shape != (T,) or \
            not positions.is_contiguous():
        raise ValueError("rope: positions must be a contiguous int64 or int32 tensor of T entries")
    if positions.get_device() != dev:
        _off_device("rope", "positions", positions, dev)
    _freqs("rope", inv_freq, dev)
    qos = None
    if q_out is None and stream is None and qs is None:
        q_out = _empty_like(q)
    else:
        q_out, qos = _result("rope", "q_out", q_out, q, stream, dev, qs is None)
    Hkv, ks, kos, kp, kop = 0, None, None, 0, 0
    if k is None:
        k_out = None
    else:
        (Tk, Hkv, Dk), ks = _rows3("rope", "k", k, dev)
        if Tk != T or Dk != D:
            raise ValueError(f"rope: k has shape {tuple(k.shape)}, q {tuple(q.shape)}")
        if k.dtype != q.dtype:
            raise TypeError(f"rope: k is {k.dtype}, not {q.dtype}")
        if k_out is None and stream is None and ks is None:
            k_out = _empty_like(k)
        else:
            k_out, kos = _result("rope", "k_out", k_out, k, stream, dev, ks is None)
        kp, kop = k.data_ptr(), k_out.data_ptr()
    if many is not None:
        pp, bits, naxes, step, ap = many
        rc = _lib.sage_rope_axes(q.data_ptr(), kp, q_out.data_ptr(), kop, dtype, T, Hq, Hkv, D, qs,
                                 ks, qos, kos, pp, bits, naxes, step, ap, inv_freq.data_ptr(),
                                 2 * inv_freq.shape[0], 1 if interleaved else 0, mscale,
                                 1 if inverse else 0, _handle(stream, current))
        if rc:
            _check(rc, "sage_rope_axes")
        return q_out, k_out
    rc = _lib.sage_rope(q.data_ptr(), kp, q_out.data_ptr(), kop, dtype, T, Hq, Hkv, D, qs, ks, qos,
                        kos, positions.data_ptr(), bits, inv_freq.data_ptr(),
                        2 * inv_freq.shape[0], 1 if interleaved else 0, mscale,
                        1 if inverse else 0, _handle(stream, current))
    if rc:
        _check(rc, "sage_rope")
    return q_out, k_out


class PagedCache:
    """A paged key/value cache over the caller's tensors (kept alive by it).
    k, v: (pages, slots, Hkv, D) ("NHD") or (pages, Hkv, slots, D) ("HND"),
    sharing their strides, channels contiguous.  fp16/bf16 tensors hold K and V
    as they are; an int8 k with a float8_e4m3fn v holds them quantised, with
    k_scale float32 (pages, Hkv, slots) and the fixed k_mean and v_scale
    float32 (Hkv, Dp), Dp = 64 if D <= 64 else 128 (kv_stats_noalloc writes
    them from a sample of keys and values).  uint8 tensors with head_dim = D hold
    four bits a channel: rows of 16 * ceil(D / 32) bytes in the place of D, the
    same k_mean and v_scale, and k_groups and v_groups float16 (pages, Hkv, slots,
    Dp / 32), a scale for each token, head and 32 channels (SAGE_Q4 in sage.h)."""

    def __init__(self, k, v, layout="NHD", k_scale=None, k_mean=None, v_scale=None, k_groups=None,
                 v_groups=None, head_dim=None):
        import torch
        lay = _layout_code(layout)
        if k.dim() != 4 or tuple(v.shape) != tuple(k.shape):
            raise ValueError(f"PagedCache: k {tuple(k.shape)} and v {tuple(v.shape)} must be 4-D "
                             "tensors of one shape")
        q8, q4 = k.dtype == torch.int8, k.dtype == torch.uint8
        if q8 and v.dtype != torch.float8_e4m3fn or q4 and v.dtype != torch.uint8 or \
                not (q8 or q4) and (k.dtype not in (torch.float16, torch.bfloat16) or
                                    v.dtype != k.dtype):
            raise TypeError(f"PagedCache: k {k.dtype} and v {v.dtype} must be both float16, both "
                            "bfloat16, int8 and float8_e4m3fn, or both uint8 (two codes a byte)")
        self.kind = Q4 if q4 else Q8 if q8 else F16 if k.dtype == torch.float16 else BF16
        self._dev = k.get_device()
        pages, width = k.shape[0], k.shape[3]
        self.D = width if head_dim is None else int(head_dim)
        if q4 and (head_dim is None or width != 16 * -(-self.D // 32)):
            raise ValueError("PagedCache: a 4-bit cache needs head_dim, and rows of "
                             f"16 * ceil(head_dim / 32) bytes, got {width} for {head_dim}")
        if not q4 and self.D != width:
            raise ValueError(f"PagedCache: head_dim is {head_dim}, the rows have {width} channels")
        slots, self.Hkv = (k.shape[2], k.shape[1]) if lay == HND else (k.shape[1], k.shape[2])
        st, page_dims = k.stride(), (2, 1) if lay == HND else (1, 2)
        for name, t in (("k", k), ("v", v)):
            _on_device("PagedCache", name, t)
            if any(n > 1 and a != b for n, a, b in zip(k.shape, t.stride(), st)):
                raise ValueError(f"PagedCache: k and v must share their strides ({k.stride()} and "
                                 f"{v.stride()})")
        if st[3] != 1 and width > 1:
            raise ValueError("PagedCache: the channels must be contiguous")
        dp = 64 if self.D <= 64 else 128
        scales = (("k_scale", k_scale, q8, torch.float32, (pages, self.Hkv, slots)),
                  ("k_mean", k_mean, q8 or q4, torch.float32, (self.Hkv, dp)),
                  ("v_scale", v_scale, q8 or q4, torch.float32, (self.Hkv, dp)),
                  ("k_groups", k_groups, q4, torch.float16, (pages, self.Hkv, slots, dp // 32)),
                  ("v_groups", v_groups, q4, torch.float16, (pages, self.Hkv, slots, dp // 32)))
        for name, t, wanted, dtype, shape in scales:
            if not wanted:
                if t is not None:
                    raise ValueError(f"PagedCache: {name} belongs to a quantised cache only"
                                     if not (q8 or q4) else
                                     f"PagedCache: {name} does not belong to this kind of cache")
                continue
            if t is None or t.dtype != dtype or tuple(t.shape) != shape or not t.is_contiguous():
                raise ValueError(f"PagedCache: {name} must be a contiguous "
                                 f"{str(dtype).replace('torch.', '')} tensor of shape {shape}")
            _on_device("PagedCache", name, t)
        self.k, self.v, self.k_scale, self.k_mean, self.v_scale = k, v, k_scale, k_mean, v_scale
        self.k_groups, self.v_groups = k_groups, v_groups
        ptr = lambda t: 0 if t is None else t.data_ptr()
        self._c = _CacheC(ptr(k), ptr(v), ptr(k_scale), ptr(k_mean), ptr(v_scale), pages, slots,
                          self.Hkv, self.D, st[0], st[page_dims[0]], st[page_dims[1]], self.kind,
                          ptr(k_groups), ptr(v_groups))
        self._ref = ctypes.byref(self._c)


class PagedBatch:
    """A batch of new tokens: int32 CUDA tensors cu_q (n + 1 offsets of the
    packed rows), kv_lens (n cached lengths, the new tokens included) and
    block_table (n, width) of page indices; max_q and max_kv bound the new
    tokens and the length of every sequence."""

    def __init__(self, cu_q, kv_lens, block_table, max_q, max_kv):
        import torch
        for name, t in (("cu_q", cu_q), ("kv_lens", kv_lens), ("block_table", block_table)):
            _on_device("PagedBatch", name, t)
            if t.dtype != torch.int32:
                raise TypeError(f"PagedBatch: {name} must be int32, got {t.dtype}")
        n = kv_lens.numel()
        if cu_q.dim() != 1 or cu_q.numel() != n + 1 or kv_lens.dim() != 1 or \
                not cu_q.is_contiguous() or not kv_lens.is_contiguous():
            raise ValueError("PagedBatch: cu_q and kv_lens must be contiguous, of n + 1 and n "
                             "entries")
        if block_table.dim() != 2 or block_table.shape[0] != n or \
                block_table.shape[1] > 1 and block_table.stride(1) != 1:
            raise ValueError(f"PagedBatch: block_table must be (n, width) with contiguous rows, "
                             f"got {tuple(block_table.shape)}")
        for name, x in (("max_q", max_q), ("max_kv", max_kv)):
            if not 0 <= int(x) <= 2 ** 31 - 1:
                raise ValueError(f"PagedBatch: {name} must be in 0..2147483647, got {x}")
        self.cu_q, self.kv_lens, self.block_table = cu_q, kv_lens, block_table
        self.nseq, self.max_q, self.max_kv = n, int(max_q), int(max_kv)
        self._calls, self._dev = {}, kv_lens.get_device()
        self._c = _BatchC(cu_q.data_ptr(), kv_lens.data_ptr(), block_table.data_ptr(), n, 0,
                          block_table.stride(0), block_table.shape[1], self.max_q, self.max_kv)

    def _rows(self, total_q):
        c = self._calls.get(total_q)                # one struct per number of rows: calls of
        if c is None:                               # several threads share the batch
            c = _BatchC.from_buffer_copy(self._c)
            c.total_q = total_q
            if len(self._calls) < 64:
                self._calls[total_q] = c
        return ctypes.byref(c)


PAGED_CLEAR_BYTES = 8192      # SAGE_PAGED_CLEAR_BYTES


def workspace_bytes_paged() -> int:
    return int(_lib.sage_workspace_bytes_paged())


def alloc_workspace_paged(device="cuda", stream=None):
    """A workspace of kv_append and attn_paged, cleared where they need it.  One
    serves any number of calls in stream order."""
    def make():
        ws = alloc_workspace(workspace_bytes_paged(), device)
        ws[:PAGED_CLEAR_BYTES].zero_()
        return ws
    return _empty_on(stream, make)


def kv_append(cache, batch, k, v, q=None, q_out=None, inv_freq=None, interleaved=False, mscale=1.0,
              ws=None, stream=None, positions=None, axes=None):
    """Writes the batch's new k and v (T, Hkv, D) into the cache.  With
    inv_freq, k is turned at each token's position first, and q (T, Hq, D), if
    given, into q_out (returned).  The rotation's positions are the tokens' places
    in their sequences, or `positions` (T,) or (A, T) with `axes`, as in rope."""
    dev, current = _device("kv_append", "k", k)
    if cache._dev != dev or batch._dev != dev:
        _off_cache("kv_append", cache, batch, dev)
    shape, ks = _rows3("kv_append", "k", k, dev)
    vshape, vs = _rows3("kv_append", "v", v, dev)
    dtype = _code16("kv_append", "k", k)
    T = shape[0]
    if shape[1] != cache.Hkv or shape[2] != cache.D or vshape != shape:
        raise ValueError(f"kv_append: k {tuple(shape)} and v {tuple(vshape)} do not fit a cache "
                         f"of {cache.Hkv} heads of {cache.D} channels")
    if v.dtype != k.dtype:
        raise TypeError(f"kv_append: v is {v.dtype}, not {k.dtype}")
    Hq, qs, qos, qp, qop = 0, None, None, 0, 0
    if q is not None:
        (Tq, Hq, Dq), qs = _rows3("kv_append", "q", q, dev)
        if Tq != T or Dq != cache.D:
            raise ValueError(f"kv_append: q has shape {tuple(q.shape)}, k {tuple(shape)}")
        if q.dtype != k.dtype:
            raise TypeError(f"kv_append: q is {q.dtype}, not {k.dtype}")
        q_out, qos = _result("kv_append", "q_out", q_out, q, stream, dev, qs is None)
        qp, qop = q.data_ptr(), q_out.data_ptr()
    fp, R = 0, 0
    if inv_freq is not None:
        _freqs("kv_append", inv_freq, dev)
        fp, R = inv_freq.data_ptr(), 2 * inv_freq.shape[0]
    ws = _workspace("kv_append", ws, stream, dev)
    if positions is not None:
        if inv_freq is None:
            raise ValueError("kv_append: positions are given without inv_freq")
        if axes is None and positions.dim() != 1:
            raise ValueError("kv_append: positions of several axes need `axes`")
        pp, bits, naxes, step, ap = _axes("kv_append", positions, axes, T, R, dev)
        rc = _lib.sage_kv_append_axes(cache._ref, batch._rows(T), k.data_ptr(), v.data_ptr(), qp,
                                      qop, dtype, Hq, ks, vs, qs, qos, pp, bits, naxes, step, ap,
                                      fp, R, 1 if interleaved else 0, mscale, ws.data_ptr(),
                                      ws.numel(), _handle(stream, current))
        if rc:
            _check(rc, "sage_kv_append_axes")
        return q_out if q is not None else None
    if axes is not None:
        raise ValueError("kv_append: axes are given without positions")
    rc = _lib.sage_kv_append(cache._ref, batch._rows(T), k.data_ptr(), v.data_ptr(), qp, qop, dtype,
                             Hq, ks, vs, qs, qos, fp, R, 1 if interleaved else 0, mscale,
                             ws.data_ptr(), ws.numel(), _handle(stream, current))
    if rc:
        _check(rc, "sage_kv_append")
    return q_out if q is not None else None


def kv_gather(cache, batch, rows, dtype=None, k_out=None, v_out=None, ws=None, stream=None):
    """The batch's `rows` tokens read back from the cache: k and v (rows, Hkv, D) of
    `dtype` (a 16-bit cache: its own), as kv_append stored them, k with its mean.
    A batch whose new tokens are all the cached ones gives whole sequences.
    Tokens without a place and of sequences beyond the batch's bounds give zeros; rows
    behind the batch's are left as they are in k_out and v_out."""
    if _torch is None:
        _bind_torch()
    dev, T = _get_device(), int(rows)
    if cache._dev != dev or batch._dev != dev:
        _off_cache("kv_gather", cache, batch, dev)
    own = cache.k.dtype if cache.kind in (F16, BF16) else None
    dtype = dtype or (k_out.dtype if k_out is not None else own)
    if dtype not in _CODES or own is not None and dtype != own:
        raise TypeError(f"kv_gather: a cache of {cache.k.dtype} does not give {dtype}")
    if T < 0:
        raise ValueError(f"kv_gather: rows must not be negative, got {rows}")
    outs, shape = [], (T, cache.Hkv, cache.D)
    for name, t in (("k_out", k_out), ("v_out", v_out)):
        st = None
        if t is None:
            t = _empty_on(stream, lambda: _torch.empty(shape, dtype=dtype, device=cache.k.device))
        else:
            got, st = _rows3("kv_gather", name, t, dev)
            if got != shape or t.dtype != dtype:
                raise ValueError(f"kv_gather: {name} must be {dtype} of shape {shape}, got {t.dtype} "
                                 f"{tuple(got)}")
        outs.append((t, st))
    ws = _workspace("kv_gather", ws, stream, dev)
    (k, ks), (v, vs) = outs
    rc = _lib.sage_kv_gather(cache._ref, batch._rows(T), k.data_ptr(), v.data_ptr(), _CODES[dtype],
                             ks, vs, ws.data_ptr(), ws.numel(), _handle(stream, _get_stream(dev)))
    if rc:
        _check(rc, "sage_kv_gather")
    return k, v


def _int32s(where, name, t, shape, dev=None):
    """A contiguous int32 tensor of this shape on the (current) device."""
    if t.dtype != _torch.int32 or tuple(t.shape) != shape or not t.is_contiguous():
        raise ValueError(f"{where}: {name} must be a contiguous int32 tensor of shape {shape}, got "
                         f"{t.dtype} {tuple(t.shape)}")
    _on_device(where, name, t, dev)


class PagePool:
    """The pages of a cache and who holds them, in the caller's int32 CUDA tensors:
    free (pages,), a stack of page indices whose next one is its last of left (1,)
    pages; table (requests, width), each request's pages; lens (requests,), its
    cached length.  `PagePool.new` makes an empty pool.  What is made here is made
    and filled on `stream` (None: the current one); nothing makes a call on another
    stream wait for that, so give the stream of the calls."""

    def __init__(self, free, left, table, lens, page_size, stream=None):
        if _torch is None:
            _bind_torch()
        if table.dim() != 2 or table.dtype != _torch.int32 or \
                table.shape[1] > 1 and table.stride(1) != 1:
            raise ValueError("PagePool: table must be an int32 (requests, width) tensor with "
                             f"contiguous rows, got {table.dtype} {tuple(table.shape)}")
        requests, width = table.shape
        _on_device("PagePool", "table", table)
        self._dev = table.get_device()
        for name, t, shape in (("free", free, (free.numel(),)), ("left", left, (1,)),
                               ("lens", lens, (requests,))):
            _int32s("PagePool", name, t, shape, self._dev)
        self.free, self.left, self.table, self.lens = free, left, table, lens
        self.page_size = int(page_size)
        self.marks = _empty_on(stream, lambda: _torch.zeros(requests, dtype=_torch.int32,
                                                            device=table.device))
        self._c = _PoolC(free.data_ptr(), left.data_ptr(), table.data_ptr(), lens.data_ptr(),
                         self.marks.data_ptr(), free.numel(), self.page_size, requests,
                         table.stride(0) if requests > 1 else width, width)
        self._ref = ctypes.byref(self._c)

    @classmethod
    def new(cls, pages, page_size, requests, max_len, device="cuda", stream=None):
        """All `pages` free (0 goes first), `requests` of up to `max_len` tokens."""
        import torch
        i32 = dict(dtype=torch.int32, device=device)
        width = max(1, -(-int(max_len) // int(page_size)))
        return cls(*_empty_on(stream, lambda: (
            torch.arange(pages - 1, -1, -1, **i32), torch.full((1,), pages, **i32),
            torch.full((requests, width), -1, **i32), torch.zeros(requests, **i32))),
            page_size, stream)


class PagedPlan:
    """The buffers of a step of n sequences with `rows` packed rows in all, at most
    max_q of one and max_kv cached tokens: cu_q, kv_lens and block_table, as the
    PagedBatch `batch`; positions and slots (int64, rows), slots as page * page_size
    + place in the page; denied, an int32 scalar, sequences that got no pages.
    Positions and slots from cu_q[n] on keep what an earlier step wrote there, whose
    pages may be another request's by now: go by cu_q.  The buffers are made and
    filled on `stream` (None: the current one); nothing makes a step on another stream
    wait for that, so give the stream of the steps."""

    def __init__(self, pool, n, rows, max_q, max_kv, stream=None):
        import torch
        n, rows, max_kv = int(n), int(rows), int(max_kv)
        if n < 0 or rows < 0 or max_kv < 0:
            raise ValueError(f"PagedPlan: sizes must not be negative (n={n}, rows={rows}, "
                             f"max_kv={max_kv})")
        width = max(1, -(-max_kv // pool.page_size))
        new = lambda *shape, dtype=torch.int32, fill=0: torch.full(
            shape, fill, dtype=dtype, device=pool.table.device)
        self.cu_q, self.kv_lens, self.denied, self.block_table, self.positions, self.slots = \
            _empty_on(stream, lambda: (
                new(n + 1), new(n), new(), new(n, width, fill=-1),
                *(new(rows, dtype=torch.int64, fill=-1) for _ in range(2))))
        self.batch = PagedBatch(self.cu_q, self.kv_lens, self.block_table, max_q, max_kv)
        self.n, self.rows = n, rows
        self._c = _PlanC(self.cu_q.data_ptr(), self.kv_lens.data_ptr(), self.block_table.data_ptr(),
                         self.positions.data_ptr(), self.slots.data_ptr(), self.denied.data_ptr(),
                         n, rows, width, width, self.batch.max_q, self.batch.max_kv)
        self._ref = ctypes.byref(self._c)


def _pool_call(where, pool, requests, ws, stream):
    """(device, requests, workspace, stream's handle) of a call on a pool."""
    dev = _get_device()
    if pool._dev != dev:
        raise ValueError(f"{where}: the pool is on cuda:{pool._dev}, the current device is "
                         f"cuda:{dev}")
    if requests.dim() != 1:
        raise ValueError(f"{where}: requests must be 1-D, got {tuple(requests.shape)}")
    _int32s(where, "requests", requests, tuple(requests.shape), dev)
    return dev, _workspace(where, ws, stream, dev), _handle(stream, _get_stream(dev))


def paged_step(pool, plan, requests, new_lens, ws=None, stream=None):
    """Makes room for new_lens (n,) more tokens of the pool's requests (n,), both
    int32: takes the pages that they need, advances the lengths and fills the plan.
    Sequences whose pages do not fit (and every later one that needs pages) are
    denied: their rows have position and slot -1, kv_lens 0, and the pool's length
    stays.  Bad requests and lengths are denied and recorded in the workspace's
    status word; of those with more than max_q new tokens, or rows behind the plan's,
    attn_paged leaves the rows unwritten.  Returns plan.batch."""
    dev, ws, handle = _pool_call("paged_step", pool, requests, ws, stream)
    if requests.shape[0] != plan.n or plan.batch._dev != dev:
        raise ValueError(f"paged_step: {requests.shape[0]} requests on cuda:{dev} for a plan of "
                         f"{plan.n} on cuda:{plan.batch._dev}")
    _int32s("paged_step", "new_lens", new_lens, (plan.n,), dev)
    rc = _lib.sage_paged_step(pool._ref, plan._ref, requests.data_ptr(), new_lens.data_ptr(),
                              ws.data_ptr(), ws.numel(), handle)
    if rc:
        _check(rc, "sage_paged_step")
    return plan.batch


def paged_trim(pool, requests, keep_lens=None, ws=None, stream=None):
    """Cuts the pool's requests (n,) to keep_lens (n,) tokens (None: they end) and
    gives the pages behind them back: drafted tokens that were rejected, finished
    requests.  A request that is not longer stays as it is."""
    dev, ws, handle = _pool_call("paged_trim", pool, requests, ws, stream)
    if keep_lens is not None:
        _int32s("paged_trim", "keep_lens", keep_lens, tuple(requests.shape), dev)
    rc = _lib.sage_paged_trim(pool._ref, requests.data_ptr(),
                              0 if keep_lens is None else keep_lens.data_ptr(), requests.shape[0],
                              ws.data_ptr(), ws.numel(), handle)
    if rc:
        _check(rc, "sage_paged_trim")


def _off_cache(where, cache, batch, dev):
    """The cache and the batch hold pointers of the device they were built on."""
    for name, index in (("cache", cache._dev), ("batch", batch._dev)):
        if index != dev:
            raise ValueError(f"{where}: the {name} is on cuda:{index}, the current device is "
                             f"cuda:{dev}")


def _workspace(where, ws, stream, dev):
    if ws is None:
        return alloc_workspace_paged("cuda", stream)
    if ws.get_device() != dev:
        _off_device(where, "ws", ws, dev)
    return ws


def attn_paged(cache, batch, q, out=None, window=0, sinks=0, sm_scale=None, lse=None, ws=None,
               stream=None):
    """Attention of the batch's new tokens, q (T, Hq, D), over the cache:
    causal, with window > 0 only the last `window` keys and the first `sinks`
    ones.  Returns out (T, Hq, D) of q's type; lse, if given, is a float32
    (T, Hq) tensor that receives the log-sum-exp of every row.  Over four bits
    batches of many rows round K and V to fp16 (sage_attn_paged in sage.h)."""
    dev, current = _device("attn_paged", "q", q)
    if cache._dev != dev or batch._dev != dev:
        _off_cache("attn_paged", cache, batch, dev)
    (T, Hq, D), qs = _rows3("attn_paged", "q", q, dev)
    dtype = _code16("attn_paged", "q", q)
    if D != cache.D:
        raise ValueError(f"attn_paged: q has {D} channels, the cache {cache.D}")
    if out is None and stream is None and qs is None:
        out = _empty_like(q)
    else:
        out, os_ = _result("attn_paged", "out", out, q, stream, dev, qs is None)
        if os_ is not None:
            raise ValueError("attn_paged: out must be contiguous")
    lp = 0
    if lse is not None:
        if lse.dtype != _torch.float32 or lse.shape != (T, Hq) or not lse.is_contiguous():
            raise ValueError("attn_paged: lse must be a contiguous float32 (T, Hq) tensor")
        _on_device("attn_paged", "lse", lse, dev)
        lp = lse.data_ptr()
    ws = _workspace("attn_paged", ws, stream, dev)
    rc = _lib.sage_attn_paged(cache._ref, batch._rows(T), q.data_ptr(), out.data_ptr(), lp, dtype,
                              Hq, qs, window, sinks, sm_scale or 0.0, ws.data_ptr(), ws.numel(),
                              _handle(stream, current))
    if rc:
        _check(rc, "sage_attn_paged")
    return out


def debug_qk_int32(qt: Quantized, seg, hq, qtile, ktile, out=None, stream=None):
    import torch
    if out is None:
        out = torch.empty(128 * 128, dtype=torch.int32, device="cuda")
    rc = _lib.sage_debug_qk_int32(ctypes.byref(qt), seg, hq, qtile, ktile, _ptr(out),
                                  _stream(stream))
    _check(rc, "sage_debug_qk_int32")
    return out.view(128, 128)


def debug_e4m3(x, out=None, stream=None):
    import torch
    if out is None:
        out = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    rc = _lib.sage_debug_e4m3(_ptr(x), _ptr(out), x.numel(), _stream(stream))
    _check(rc, "sage_debug_e4m3")
    return out


def debug_pv_accum(p8, v8, status, out=None, stream=None):
    """sum_t P~_t V~_t^T through the attention kernel's own FP8 PV instructions.
    p8: uint8 CUDA tensor [ntiles, 128, 128] (e4m3 codes, key fastest);
    v8: uint8 CUDA tensor [ntiles, Dp, 128] (channel-major); status: a 4-byte
    CUDA tensor the call clears (read with device_status).  Returns fp32
    [128, Dp]."""
    import torch
    for name, t in (("p8", p8), ("v8", v8)):
        if not (t.is_cuda and t.is_contiguous() and t.dtype == torch.uint8):
            raise ValueError(f"{name} must be a contiguous uint8 CUDA tensor")
    ntiles, dp = v8.shape[0], v8.shape[1]
    if tuple(p8.shape) != (ntiles, 128, 128) or tuple(v8.shape) != (ntiles, dp, 128):
        raise ValueError("p8 must be [ntiles,128,128] and v8 [ntiles,Dp,128]")
    if out is None:
        out = torch.empty(128, dp, dtype=torch.float32, device=p8.device)
    rc = _lib.sage_debug_pv_accum(_ptr(p8), _ptr(v8), ntiles, dp, _ptr(out), _ptr(status),
                                  _stream(stream))
    _check(rc, "sage_debug_pv_accum")
    return out


def kv_stats_noalloc(k, v, layout, k_mean, s_v, stream=None):
    """K channel means and V channel scales with no device allocation at all:
    the scratch is a static array inside the library (B*Hkv*Dp <= 16384).
    k_mean and s_v are caller-owned contiguous fp32 CUDA tensors of at least
    B*Hkv*Dp elements (Dp = 64 if D <= 64 else 128).  kv_stats_noalloc_status
    reports a failure on the device."""
    import torch
    if k.dim() != 4 or tuple(v.shape) != tuple(k.shape):
        raise ValueError(f"kv_stats_noalloc: k {tuple(k.shape)} and v {tuple(v.shape)} must be "
                         "4-D tensors of one shape")
    lay = _layout_code(layout)
    if lay == HND:
        B, Hkv, Lk, D = k.shape
    else:
        B, Lk, Hkv, D = k.shape
    need = B * Hkv * (64 if D <= 64 else 128)
    for name, t in (("k_mean", k_mean), ("s_v", s_v)):
        if t.dtype != torch.float32 or not t.is_contiguous():
            raise ValueError(f"kv_stats_noalloc: {name} must be a contiguous float32 tensor")
        if t.numel() < need:
            raise ValueError(f"kv_stats_noalloc: {name} has {t.numel()} elements, needs {need}")
    _require_dense("kv_stats_noalloc", k, k, v)
    for name, t in (("k_mean", k_mean), ("s_v", s_v)):
        if not t.is_cuda:
            raise ValueError(f"kv_stats_noalloc: {name} is not on a CUDA device")
    rc = _lib.sage_kv_stats_noalloc(_ptr(k), _ptr(v), _dtype_code(k), lay, B, Hkv, Lk, D,
                                    _ptr(k_mean), _ptr(s_v), _stream(stream))
    _check(rc, "sage_kv_stats_noalloc")
    return k_mean, s_v


def workspace_bytes_varlen_host(nseq, total_q, total_k, Hq, Hkv, D, chunk_kv_heads=0) -> int:
    return int(_lib.sage_workspace_bytes_varlen_host(nseq, total_q, total_k, Hq, Hkv, D,
                                                     int(chunk_kv_heads)))


def attn_fwd_varlen_host(q, k, v, out, cu_q, cu_k, max_q, max_k, is_causal=False,
                         sm_scale=None, chunk_kv_heads=0, ws=None, stream=None):
    """Packed-sequence attention on host tensors (q, k, v packed (T, H, D),
    page-locked for overlap; out float32 of q's shape; cu_q and cu_k int32
    host tensors of nseq + 1 offsets): the library copies chunks of kv heads
    in, computes them and copies the output back, pipelined.  `stream`
    completes when `out` is filled."""
    import torch
    for name, t in (("q", q), ("k", k), ("v", v), ("out", out), ("cu_q", cu_q),
                    ("cu_k", cu_k)):
        if t.is_cuda or not t.is_contiguous():
            raise ValueError(f"attn_fwd_varlen_host: {name} must be a contiguous host tensor")
    if k.dtype != q.dtype or v.dtype != q.dtype:
        raise TypeError("attn_fwd_varlen_host: q, k and v must share one dtype")
    if cu_q.dtype != torch.int32 or cu_k.dtype != torch.int32:
        raise TypeError("attn_fwd_varlen_host: cu_q and cu_k must be int32")
    if q.dim() != 3 or k.dim() != 3 or tuple(v.shape) != tuple(k.shape):
        raise ValueError("attn_fwd_varlen_host: q, k, v must be packed (T, H, D), v like k")
    if out.dtype != torch.float32 or tuple(out.shape) != tuple(q.shape):
        raise ValueError("attn_fwd_varlen_host: out must be float32 with q's shape")
    if cu_q.numel() != cu_k.numel() or cu_q.numel() < 2:
        raise ValueError("attn_fwd_varlen_host: cu_q and cu_k need the same nseq + 1 >= 2 entries")
    total_q, Hq, D = q.shape
    total_k, Hkv, _ = k.shape
    nseq = cu_q.numel() - 1
    if ws is None:
        ws = alloc_workspace(workspace_bytes_varlen_host(nseq, total_q, total_k, Hq, Hkv, D,
                                                         chunk_kv_heads))
    rc = _lib.sage_attn_fwd_varlen_host(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(cu_q),
                                        _ptr(cu_k), nseq, total_q, total_k, int(max_q),
                                        int(max_k), Hq, Hkv, D, int(bool(is_causal)),
                                        float(sm_scale or 0.0), _dtype_code(q),
                                        int(chunk_kv_heads), _ptr(ws), ws.numel(),
                                        _stream(stream))
    _check(rc, "sage_attn_fwd_varlen_host")
    return out


def debug_tc_rate(kind: int, n_mma: int, status, stream=None):
    """Enqueues n_mma back-to-back M=128 N=128 tcgen05 MMAs per SM (kind 0:
    fp16 K=16, kind 1: e4m3 K=32); time it with events on `stream`."""
    _check(_lib.sage_debug_tc_rate(int(kind), int(n_mma), _ptr(status), _stream(stream)),
           "sage_debug_tc_rate")


def kv_stats_noalloc_status(stream=None) -> int:
    """Device status of the last kv_stats_noalloc call on this device."""
    return int(_lib.sage_kv_stats_noalloc_status(_stream(stream)))


def set_fault(skip_kv_tile: int = -1, timeout_ns: int = 0, launches: int = -1):
    """Failure injection: attention launches skip key/value tile skip_kv_tile
    (-1: off) and give up waiting after timeout_ns; launches >= 0 limits the
    fault to that many launches."""
    _lib.sage_debug_set_fault_launches(int(launches))
    _lib.sage_debug_set_fault(int(skip_kv_tile), int(timeout_ns))


def set_prologue_launches(launches: int = 0):
    """Test hook: 1 or 2 prologue launches, 0 to choose by size."""
    _lib.sage_debug_set_prologue_launches(int(launches))


def set_host_fail_chunk(chunk: int = -1):
    """Test hook: the host-buffer calls fail at chunk `chunk` (-1: off)."""
    _lib.sage_debug_set_host_fail_chunk(int(chunk))


def device_status(ws, stream=None) -> int:
    return int(_lib.sage_device_status(_ptr(ws), _stream(stream)))


def ws_view(qt: Quantized, field: str, dtype, shape):
    """A torch view of one workspace buffer (for tests and inspection)."""
    import torch
    ws = qt._ws
    off = getattr(qt, field) - ws.data_ptr()
    n = 1
    for s in shape:
        n *= s
    nbytes = n * torch.tensor([], dtype=dtype).element_size()
    return ws[off:off + nbytes].view(dtype).view(*shape)
