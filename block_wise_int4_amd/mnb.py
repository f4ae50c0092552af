"""Thin Python binding of libmnb (include/mnb.h).

Argument marshalling only: every step of the computation runs in the HIP
kernels behind the C ABI.  The functions keep the C names; device buffers are
torch CUDA tensors (or raw integer device addresses), and the stream is the
current torch stream unless one is passed.  A non-OK status raises MnbError
with the library's reason.  There is no fallback: if the library is missing
the import fails.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Union

try:                       # device memory and streams; the host-only calls work without it
    import torch
except ImportError:
    torch = None
try:                       # the current stream's handle without building a stream object (2.8 us a call)
    from torch._C import _cuda_getCurrentRawStream as _raw_stream, _cuda_getDevice as _current_device
    from torch.cuda import is_initialized as _initialized
except ImportError:        # private names: without them torch's public call gives the stream
    _raw_stream = None

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "lib", "libmnb.so")

MNB_OK = 0
MNB_ERR_INVALID_ARGUMENT = 1
MNB_ERR_UNSUPPORTED = 2
MNB_ERR_DEVICE = 3
MNB_F32 = 0
MNB_F16 = 1
MNB_BIAS_FUSED = 0
MNB_BIAS_AFTER_ROUND = 1
MNB_NORM_VALUES = 0
MNB_NORM_CODES_F16 = 1
MNB_NORM_CODES_I8 = 2

EXPORTS = ("mnb_repacked_bytes", "mnb_repacked_layout", "mnb_repack", "mnb_gemv",
           "mnb_gemv_gate_up_swiglu", "mnb_gemm_workspace_bytes", "mnb_gemm_workspace_bytes_for", "mnb_gemm",
           "mnb_gemm_bias",
           "mnb_act_order_permutation", "mnb_repack_act_order", "mnb_gemm_act_order_workspace_bytes",
           "mnb_gemm_act_order", "mnb_gemm_group_indices", "mnb_gemm_accuracy4_workspace_bytes", "mnb_gemm_accuracy4",
           "mnb_gemm_accuracy4_noalloc", "mnb_gemm_accuracy4_codes", "mnb_rms_norm",
           "mnb_kv4_cache_bytes", "mnb_kv4_append", "mnb_kv4_read", "mnb_attention_kv4_workspace_bytes",
           "mnb_attention_kv4",
           "mnb_unpack_debug", "mnb_debug_prefill_rows", "mnb_status_string", "mnb_last_error", "mnb_last_variant")


class MnbError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__("%s: %s" % (_status_name(status), message))
        self.status = status


class mnb_weight_desc(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int64), ("k", ctypes.c_int64), ("group_size", ctypes.c_int32),
                ("has_zero_points", ctypes.c_int32), ("scale_dtype", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class mnb_kv4_desc(ctypes.Structure):
    _fields_ = [("q_heads", ctypes.c_int32), ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("group_size", ctypes.c_int32), ("page_size", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("num_pages", ctypes.c_int64)]


class mnb_layout(ctypes.Structure):
    _fields_ = [(name, ctypes.c_int64) for name in (
        "tiles", "chunks", "groups_per_chunk", "codes_offset", "codes_bytes", "scales_offset",
        "scales_bytes", "zero_points_offset", "zero_points_bytes", "range_flags_offset",
        "range_flags_bytes", "total_bytes")]


def _hip_runtimes_mapped():
    """Paths of the HIP runtime libraries mapped into this process."""
    try:
        with open("/proc/self/maps") as f:
            return sorted({line.split()[-1] for line in f if "libamdhip64" in line})
    except OSError:
        return []


def _load():
    # torch brings its own HIP runtime.  It must be the one libmnb binds to:
    # device pointers and streams are only meaningful inside one runtime, so
    # torch is loaded first and libmnb's libamdhip64.so.7 dependency resolves
    # to the copy already in the process.
    try:
        import torch  # noqa: F401
    except ImportError:
        pass
    if not os.path.exists(LIB_PATH):
        raise ImportError("libmnb.so is not built (%s); run `python -m block_wise_int4_amd.build`"
                          % LIB_PATH)
    lib = ctypes.CDLL(LIB_PATH)
    P = ctypes.c_void_p
    D = ctypes.POINTER(mnb_weight_desc)
    KV = ctypes.POINTER(mnb_kv4_desc)
    i32, i64, sz, f32 = ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
    sig = {
        "mnb_repacked_bytes": (sz, [D]),
        "mnb_repacked_layout": (ctypes.c_int, [D, ctypes.POINTER(mnb_layout)]),
        "mnb_repack": (ctypes.c_int, [D, P, P, P, P, P]),
        "mnb_gemv": (ctypes.c_int, [D, P, P, i32, P, P]),
        "mnb_gemv_gate_up_swiglu": (ctypes.c_int, [D, P, P, P, i32, P, P]),
        "mnb_gemm_workspace_bytes": (sz, [D, i64]),
        "mnb_gemm_workspace_bytes_for": (sz, [D, i64, i32]),
        "mnb_gemm": (ctypes.c_int, [D, P, P, i64, i32, P, P, sz, P]),
        "mnb_gemm_bias": (ctypes.c_int, [D, P, P, i64, i32, P, i64, i32, P, P, sz, P]),
        "mnb_act_order_permutation": (ctypes.c_int, [D, P, P]),
        "mnb_repack_act_order": (ctypes.c_int, [D, P, P, P, P, P, P]),
        "mnb_gemm_act_order_workspace_bytes": (sz, [D, i64, i32]),
        "mnb_gemm_act_order": (ctypes.c_int, [D, P, P, i64, i32, P, P, P, sz, P]),
        "mnb_gemm_group_indices": (ctypes.c_int, [D, P, P, i64, i32, P, P, i64, i32, P, P]),
        "mnb_gemm_accuracy4_workspace_bytes": (sz, [D, i64]),
        "mnb_gemm_accuracy4": (ctypes.c_int, [D, P, P, i64, P, P, P, sz, P]),
        "mnb_gemm_accuracy4_noalloc": (ctypes.c_int, [D, P, P, i64, P, P, P]),
        "mnb_gemm_accuracy4_codes": (ctypes.c_int, [D, P, P, P, i64, P, P, P]),
        "mnb_rms_norm": (ctypes.c_int, [P, i64, P, i64, P, i64, i64, i32, f32, i32, P, P, P, P]),
        "mnb_kv4_cache_bytes": (sz, [KV]),
        "mnb_kv4_append": (ctypes.c_int, [KV, P, P, i64, P, P, i64, i64, i32, P, i64, P, i64, P, i64, P, P, i64,
                                          i32, i32, P, P]),
        "mnb_kv4_read": (ctypes.c_int, [KV, P, P, i64, P, P, i64, i64, i32, P, P, P]),
        "mnb_attention_kv4_workspace_bytes": (sz, [KV, i64, i64, i64, i64]),
        "mnb_attention_kv4": (ctypes.c_int, [KV, P, P, i64, P, P, i64, i64, i64, i64, i32, P, i64, f32, i32, i64, P,
                                             P, P, sz, P]),
        "mnb_unpack_debug": (ctypes.c_int, [D, P, P, P, P]),
        "mnb_debug_prefill_rows": (ctypes.c_int32, [ctypes.c_int32]),
        "mnb_status_string": (ctypes.c_char_p, [ctypes.c_int]),
        "mnb_last_error": (ctypes.c_char_p, []),
        "mnb_last_variant": (ctypes.c_char_p, []),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    runtimes = _hip_runtimes_mapped()
    if len(runtimes) > 1:
        raise ImportError("two HIP runtimes are loaded (%s); import torch before loading libmnb"
                          % ", ".join(runtimes))
    return lib


lib = _load()


def _status_name(s: int) -> str:
    return lib.mnb_status_string(s).decode()


def _check(status: int) -> None:
    if status != MNB_OK:
        raise MnbError(status, lib.mnb_last_error().decode())


Ptr = Union[int, None, "torch.Tensor"]


def _ptr(x: Ptr):
    if x is None:
        return None
    if isinstance(x, int):
        return ctypes.c_void_p(x)
    if not x.is_cuda:
        raise ValueError("device tensor expected")
    if not x.is_contiguous():
        raise ValueError("contiguous tensor expected")
    return ctypes.c_void_p(x.data_ptr())


def _stream(stream):
    if stream is None:
        if _raw_stream is not None and _initialized():
            return _raw_stream(_current_device())
        stream = torch.cuda.current_stream()
    if isinstance(stream, int):
        return ctypes.c_void_p(stream)
    return ctypes.c_void_p(stream.cuda_stream)


def _dtype_code(t) -> int:
    if t.dtype is torch.float16:
        return MNB_F16
    if t.dtype is torch.float32:
        return MNB_F32
    raise ValueError("fp16 or fp32 tensor expected, got %s" % t.dtype)


def desc(n: int, k: int, group_size: int, has_zero_points: bool, scale_dtype: int) -> mnb_weight_desc:
    return mnb_weight_desc(n, k, group_size, int(bool(has_zero_points)), scale_dtype, 0)


# ---- the C entry points -----------------------------------------------------

def mnb_repacked_bytes(w: mnb_weight_desc) -> int:
    size = lib.mnb_repacked_bytes(ctypes.byref(w))
    if size == 0:
        raise MnbError(MNB_ERR_INVALID_ARGUMENT, lib.mnb_last_error().decode())
    return int(size)


def mnb_repacked_layout(w: mnb_weight_desc) -> dict:
    out = mnb_layout()
    _check(lib.mnb_repacked_layout(ctypes.byref(w), ctypes.byref(out)))
    return {name: getattr(out, name) for name, _ in mnb_layout._fields_}


def mnb_repack(w: mnb_weight_desc, packed: Ptr, scales: Ptr, zero_points: Ptr, repacked: Ptr,
               stream=None) -> None:
    _check(lib.mnb_repack(ctypes.byref(w), _ptr(packed), _ptr(scales), _ptr(zero_points),
                          _ptr(repacked), _stream(stream)))


def mnb_gemv(w: mnb_weight_desc, repacked: Ptr, a, y, a_dtype: Optional[int] = None,
             stream=None) -> None:
    dt = _dtype_code(a) if a_dtype is None else a_dtype
    _check(lib.mnb_gemv(ctypes.byref(w), _ptr(repacked), _ptr(a), dt, _ptr(y), _stream(stream)))


def mnb_gemv_gate_up_swiglu(w: mnb_weight_desc, gate_repacked: Ptr, up_repacked: Ptr, a, y,
                            a_dtype: Optional[int] = None, stream=None) -> None:
    dt = _dtype_code(a) if a_dtype is None else a_dtype
    _check(lib.mnb_gemv_gate_up_swiglu(ctypes.byref(w), _ptr(gate_repacked), _ptr(up_repacked),
                                       _ptr(a), dt, _ptr(y), _stream(stream)))


def mnb_gemm_workspace_bytes(w: mnb_weight_desc, m: int) -> int:
    return int(lib.mnb_gemm_workspace_bytes(ctypes.byref(w), m))


def mnb_gemm_workspace_bytes_for(w: mnb_weight_desc, m: int, a_dtype: int) -> int:
    return int(lib.mnb_gemm_workspace_bytes_for(ctypes.byref(w), m, a_dtype))


def mnb_gemm(w: mnb_weight_desc, repacked: Ptr, a, m: int, y, workspace: Ptr = None,
             workspace_bytes: Optional[int] = None, a_dtype: Optional[int] = None,
             stream=None) -> None:
    dt = _dtype_code(a) if a_dtype is None else a_dtype
    if workspace_bytes is None:
        workspace_bytes = 0 if workspace is None or isinstance(workspace, int) else \
            workspace.numel() * workspace.element_size()
    _check(lib.mnb_gemm(ctypes.byref(w), _ptr(repacked), _ptr(a), m, dt, _ptr(y),
                        _ptr(workspace), workspace_bytes, _stream(stream)))


def mnb_gemm_bias(w: mnb_weight_desc, repacked: Ptr, a, m: int, bias, bias_row_stride: int,
                  bias_mode: int, y, workspace: Ptr = None, workspace_bytes: Optional[int] = None,
                  a_dtype: Optional[int] = None, stream=None) -> None:
    dt = _dtype_code(a) if a_dtype is None else a_dtype
    if workspace_bytes is None:
        workspace_bytes = 0 if workspace is None or isinstance(workspace, int) else \
            workspace.numel() * workspace.element_size()
    _check(lib.mnb_gemm_bias(ctypes.byref(w), _ptr(repacked), _ptr(a), m, dt, _ptr(bias),
                             bias_row_stride, bias_mode, _ptr(y), _ptr(workspace), workspace_bytes,
                             _stream(stream)))


def mnb_act_order_permutation(w: mnb_weight_desc, g_idx):
    """Host: the act-order permutation of k for a g_idx (numpy int32 [K])."""
    import numpy as np
    g = np.ascontiguousarray(g_idx, np.int32)
    perm = np.empty(g.size, dtype=np.int32)
    _check(lib.mnb_act_order_permutation(ctypes.byref(w), g.ctypes.data_as(ctypes.c_void_p),
                                         perm.ctypes.data_as(ctypes.c_void_p)))
    return perm


def mnb_repack_act_order(w: mnb_weight_desc, packed: Ptr, scales: Ptr, zero_points: Ptr, perm: Ptr,
                         repacked: Ptr, stream=None) -> None:
    _check(lib.mnb_repack_act_order(ctypes.byref(w), _ptr(packed), _ptr(scales), _ptr(zero_points),
                                    _ptr(perm), _ptr(repacked), _stream(stream)))


def mnb_gemm_act_order_workspace_bytes(w: mnb_weight_desc, m: int, a_dtype: int = MNB_F16) -> int:
    return int(lib.mnb_gemm_act_order_workspace_bytes(ctypes.byref(w), m, a_dtype))


def mnb_gemm_act_order(w: mnb_weight_desc, repacked: Ptr, a, m: int, perm: Ptr, y, workspace: Ptr,
                       workspace_bytes: Optional[int] = None, a_dtype: Optional[int] = None,
                       stream=None) -> None:
    dt = _dtype_code(a) if a_dtype is None else a_dtype
    if workspace_bytes is None:
        workspace_bytes = 0 if workspace is None or isinstance(workspace, int) else \
            workspace.numel() * workspace.element_size()
    _check(lib.mnb_gemm_act_order(ctypes.byref(w), _ptr(repacked), _ptr(a), m, dt, _ptr(perm), _ptr(y),
                                  _ptr(workspace), workspace_bytes, _stream(stream)))


def mnb_gemm_group_indices(w: mnb_weight_desc, repacked: Ptr, a, m: int, g_idx: Ptr, y, bias=None,
                           bias_row_stride: int = 0, bias_mode: int = MNB_BIAS_FUSED,
                           a_dtype: Optional[int] = None, stream=None) -> None:
    dt = _dtype_code(a) if a_dtype is None else a_dtype
    _check(lib.mnb_gemm_group_indices(ctypes.byref(w), _ptr(repacked), _ptr(a), m, dt, _ptr(g_idx), _ptr(bias),
                                      bias_row_stride, bias_mode, _ptr(y), _stream(stream)))


def mnb_gemm_accuracy4_workspace_bytes(w: mnb_weight_desc, m: int) -> int:
    return int(lib.mnb_gemm_accuracy4_workspace_bytes(ctypes.byref(w), m))


def mnb_gemm_accuracy4(w: mnb_weight_desc, repacked: Ptr, a, m: int, bias, y, workspace: Ptr = None,
                       workspace_bytes: Optional[int] = None, stream=None) -> None:
    if workspace_bytes is None:
        workspace_bytes = 0 if workspace is None or isinstance(workspace, int) else \
            workspace.numel() * workspace.element_size()
    _check(lib.mnb_gemm_accuracy4(ctypes.byref(w), _ptr(repacked), _ptr(a), m, _ptr(bias), _ptr(y),
                                  _ptr(workspace), workspace_bytes, _stream(stream)))


MNB_NOALLOC_SCRATCH_BYTES = 32 << 20


def mnb_gemm_accuracy4_noalloc(w: mnb_weight_desc, repacked: Ptr, a, m: int, bias, y, stream=None) -> None:
    _check(lib.mnb_gemm_accuracy4_noalloc(ctypes.byref(w), _ptr(repacked), _ptr(a), m, _ptr(bias), _ptr(y),
                                          _stream(stream)))


def mnb_gemm_accuracy4_codes(w: mnb_weight_desc, repacked: Ptr, codes: Ptr, scales: Ptr, m: int, bias, y,
                             stream=None) -> None:
    _check(lib.mnb_gemm_accuracy4_codes(ctypes.byref(w), _ptr(repacked), _ptr(codes), _ptr(scales), m, _ptr(bias),
                                        _ptr(y), _stream(stream)))


# ---- between the products ---------------------------------------------------
# These calls are short on the device: the checks of a tensor are single
# comparisons, and only a failing one builds a message.

def _addr(x, name: str) -> Optional[int]:
    """Address of a dense device tensor (or None, or an address)."""
    if x is None or type(x) is int:
        return x
    if not x.is_cuda or not x.is_contiguous():
        raise ValueError("%s: contiguous device tensor expected" % name)
    return x.data_ptr()


def _refuse(tensors) -> None:
    """Raises for the first of (tensor, name, dtype, shape) that is not as it should be."""
    for x, name, dtype, shape in tensors:
        if x.dtype is not dtype:
            raise ValueError("%s: %s expected, got %s" % (name, dtype, x.dtype))
        if x.shape != shape:
            raise ValueError("%s: shape %s expected, got %s" % (name, tuple(shape), tuple(x.shape)))


def _rows2(x, name: str):
    """Address and row stride of an [m, k] tensor whose rows are dense."""
    stride, shape = x.stride(), x.shape
    if not x.is_cuda or (stride[1] != 1 and shape[1] > 1):
        raise ValueError("%s: device tensor with dense rows expected" % name)
    return x.data_ptr(), stride[0] if shape[0] > 1 else shape[1]


def _rows3(x, heads: int, dim: int, name: str):
    """The same for [tokens, heads, dim]: a token's heads and dims are dense."""
    stride = x.stride()
    if not x.is_cuda or stride[2] != 1 or (stride[1] != dim and heads > 1):
        raise ValueError("%s: device tensor with dense rows expected" % name)
    return x.data_ptr(), stride[0] if x.shape[0] > 1 else heads * dim


def mnb_rms_norm(x, weight, out, eps: float, residual=None, residual_out=None, scales=None, stream=None) -> None:
    """x, residual [m, k] (rows may be strided), out and residual_out [m, k].  Without `scales` out receives the
    values; with it (fp32 [m]) the 8-bit codes, as int8 or as fp16 integers by out's type."""
    shape, dtype = x.shape, x.dtype
    m, k = shape
    kind, want = MNB_NORM_VALUES, dtype
    if scales is not None:
        kind, want = (MNB_NORM_CODES_I8, torch.int8) if out.dtype is torch.int8 else (MNB_NORM_CODES_F16, torch.float16)
        if scales.dtype is not torch.float32 or scales.shape != (m,):
            _refuse(((scales, "scales", torch.float32, (m,)),))
    if out.dtype is not want or out.shape != shape or weight.dtype is not dtype or weight.shape != (k,):
        _refuse(((out, "out", want, shape), (weight, "weight", dtype, (k,))))
    xp, xs = _rows2(x, "x")
    rp, rs = None, 0
    if residual is not None:
        if residual.dtype is not dtype or residual.shape != shape:
            _refuse(((residual, "residual", dtype, shape),))
        rp, rs = _rows2(residual, "residual")
    if residual_out is not None and (residual_out.dtype is not dtype or residual_out.shape != shape):
        _refuse(((residual_out, "residual_out", dtype, shape),))
    st = lib.mnb_rms_norm(xp, xs, rp, rs, _addr(weight, "weight"), m, k, _dtype_code(x), eps, kind, _addr(out, "out"),
                          _addr(scales, "scales"), _addr(residual_out, "residual_out"), _stream(stream))
    if st:
        _check(st)


def kv4_desc(q_heads: int, kv_heads: int, head_dim: int, group_size: int, page_size: int,
             num_pages: int) -> mnb_kv4_desc:
    return mnb_kv4_desc(q_heads, kv_heads, head_dim, group_size, page_size, 0, num_pages)


def mnb_kv4_cache_bytes(c: mnb_kv4_desc) -> int:
    size = lib.mnb_kv4_cache_bytes(ctypes.byref(c))
    if size == 0:
        raise MnbError(MNB_ERR_INVALID_ARGUMENT, lib.mnb_last_error().decode())
    return int(size)


def _sequences(c, cache, table, kv_len, q_start):
    """Descriptor, cache, table, table stride, lengths, offsets and batch of a call, after a look at their types and sizes."""
    i32 = torch.int32
    batch = kv_len.shape[0]
    if table.dtype is not i32 or kv_len.dtype is not i32 or (q_start is not None and q_start.dtype is not i32):
        raise ValueError("block_table, kv_len and q_start: int32 expected")
    if table.shape[0] != batch or (q_start is not None and q_start.shape[0] != batch + 1):
        raise ValueError("block_table, kv_len and q_start: one row, length and offset (and one more) per sequence")
    d = ctypes.byref(c)
    if cache.numel() * cache.element_size() < lib.mnb_kv4_cache_bytes(d):
        raise ValueError("cache: %d bytes expected" % mnb_kv4_cache_bytes(c))
    # a row's length is its pitch: of a slice of a wider table the kernels would take the entries beside it
    return d, _addr(cache, "cache"), _addr(table, "block_table"), table.shape[1], _addr(kv_len, "kv_len"), \
        _addr(q_start, "q_start"), batch


def mnb_kv4_append(c: mnb_kv4_desc, cache, k, v, block_table, kv_len, q_start=None, cos=None, sin=None,
                   rotary_dim: int = 0, interleaved: bool = False, q=None, q_out=None, stream=None) -> None:
    """k, v [tokens, kv_heads, head_dim] and q [tokens, q_heads, head_dim], tokens may be strided."""
    d, cp, tp, ts, lp, sp, batch = _sequences(c, cache, block_table, kv_len, q_start)
    dtype, n, D, H = k.dtype, k.shape[0], c.head_dim, c.kv_heads
    shape = (n, H, D)
    if k.shape != shape or v.dtype is not dtype or v.shape != shape:
        _refuse(((k, "k", dtype, shape), (v, "v", dtype, shape)))
    kp, ks = _rows3(k, H, D, "k")
    vp, vs = _rows3(v, H, D, "v")
    qp, qs, rows = None, 0, 0
    if q is not None:
        H = c.q_heads
        shape = (n, H, D)
        if q.dtype is not dtype or q.shape != shape or (q_out is not None and (q_out.dtype is not dtype or q_out.shape != shape)):
            _refuse(((q, "q", dtype, shape), (q_out, "q_out", dtype, shape)))
        qp, qs = _rows3(q, H, D, "q")
    if cos is not None:
        rows = cos.shape[0]
        shape = (rows, rotary_dim // 2)
        f32 = torch.float32
        if cos.dtype is not f32 or cos.shape != shape or (sin is not None and (sin.dtype is not f32 or sin.shape != shape)):
            _refuse(((cos, "cos", f32, shape), (sin, "sin", f32, shape)))
    st = lib.mnb_kv4_append(d, cp, tp, ts, lp, sp, batch, n, _dtype_code(k), qp, qs, kp, ks, vp, vs, _addr(cos, "cos"),
                            _addr(sin, "sin"), rows, rotary_dim, 1 if interleaved else 0, _addr(q_out, "q_out"),
                            _stream(stream))
    if st:
        _check(st)


def mnb_kv4_read(c: mnb_kv4_desc, cache, block_table, kv_len, q_start, k_out=None, v_out=None, stream=None) -> None:
    """k_out, v_out [tokens, kv_heads, head_dim]; either may be None."""
    d, cp, tp, ts, lp, sp, batch = _sequences(c, cache, block_table, kv_len, q_start)
    some = k_out if k_out is not None else v_out
    if some is None:
        return
    dtype = some.dtype
    shape = (some.shape[0], c.kv_heads, c.head_dim)
    for x in (k_out, v_out):
        if x is not None and (x.dtype is not dtype or x.shape != shape):
            _refuse(((x, "k_out and v_out", dtype, shape),))
    st = lib.mnb_kv4_read(d, cp, tp, ts, lp, sp, batch, shape[0], _dtype_code(some), _addr(k_out, "k_out"),
                          _addr(v_out, "v_out"), _stream(stream))
    if st:
        _check(st)


def mnb_attention_kv4_workspace_bytes(c: mnb_kv4_desc, batch: int, tokens: int, max_q: int, max_kv: int) -> int:
    return int(lib.mnb_attention_kv4_workspace_bytes(ctypes.byref(c), batch, tokens, max_q, max_kv))


def mnb_attention_kv4(c: mnb_kv4_desc, cache, q, block_table, kv_len, q_start, max_q: int, max_kv: int, out,
                      scale: float, causal: bool = True, window: int = 0, lse=None, workspace: Ptr = None,
                      workspace_bytes: Optional[int] = None, stream=None) -> None:
    """q [tokens, q_heads, head_dim] (tokens may be strided), out the same, lse fp32 [tokens, q_heads]."""
    d, cp, tp, ts, lp, sp, batch = _sequences(c, cache, block_table, kv_len, q_start)
    dtype, n, H, D = q.dtype, q.shape[0], c.q_heads, c.head_dim
    shape = (n, H, D)
    if q.shape != shape or out.dtype is not dtype or out.shape != shape:
        _refuse(((q, "q", dtype, shape), (out, "out", dtype, shape)))
    if lse is not None and (lse.dtype is not torch.float32 or lse.shape != (n, H)):
        _refuse(((lse, "lse", torch.float32, (n, H)),))
    if workspace_bytes is None:
        workspace_bytes = 0 if workspace is None or type(workspace) is int else \
            workspace.numel() * workspace.element_size()
    qp, qs = _rows3(q, H, D, "q")
    st = lib.mnb_attention_kv4(d, cp, tp, ts, lp, sp, batch, n, max_q, max_kv, _dtype_code(q), qp, qs, scale,
                               1 if causal else 0, window, _addr(out, "out"), _addr(lse, "lse"),
                               _addr(workspace, "workspace"), workspace_bytes, _stream(stream))
    if st:
        _check(st)


def mnb_unpack_debug(w: mnb_weight_desc, repacked: Ptr, codes: Ptr, w_f32: Ptr, stream=None) -> None:
    _check(lib.mnb_unpack_debug(ctypes.byref(w), _ptr(repacked), _ptr(codes), _ptr(w_f32),
                                _stream(stream)))


def mnb_debug_prefill_rows(rows: int) -> int:
    return lib.mnb_debug_prefill_rows(rows)


def mnb_status_string(s: int) -> str:
    return _status_name(s)


def mnb_last_error() -> str:
    return lib.mnb_last_error().decode()


def mnb_last_variant() -> str:
    return lib.mnb_last_variant().decode()


# ---- convenience over torch tensors (allocation only) -----------------------

class QuantWeight:
    """A repacked weight resident on the device, plus its descriptor."""

    def __init__(self, desc_: mnb_weight_desc, repacked):
        self.desc = desc_
        self.repacked = repacked

    @property
    def n(self) -> int:
        return self.desc.n

    @property
    def k(self) -> int:
        return self.desc.k


def repack(packed, scales, zero_points, n: int, k: int, group_size: int, stream=None) -> QuantWeight:
    """Allocate the repacked buffer (torch) and run mnb_repack into it."""
    import torch
    d = desc(n, k, group_size, zero_points is not None, _dtype_code(scales))
    out = torch.empty(mnb_repacked_bytes(d), dtype=torch.uint8, device=packed.device)
    mnb_repack(d, packed, scales, zero_points, out, stream)
    return QuantWeight(d, out)
