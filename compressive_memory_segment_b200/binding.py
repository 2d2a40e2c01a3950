"""Python binding of libinfini_attn.so (the C ABI in include/infini_attn.h).

Argument marshalling only: every step of the layer runs in the library's CUDA
kernels. torch supplies device memory and streams. There is no fallback: if the
compiled library is missing this module raises ImportError at import time.

The functions keep the C names. ``forward`` is a convenience wrapper that
allocates the outputs with torch and calls ``infini_attn_forward_ws``.
"""
from __future__ import annotations

import ctypes
import functools
import os
import struct
from typing import Optional

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "lib", "libinfini_attn.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        "libinfini_attn.so is not built (%s); run `python -m compressive_memory_segment_b200.build` "
        "or __graft_entry__.build()" % LIB_PATH)

_lib = ctypes.CDLL(LIB_PATH)

INFINI_F32, INFINI_BF16 = 0, 1
INFINI_OK = 0
INFINI_ERR_NULL, INFINI_ERR_SHAPE, INFINI_ERR_UNSUPPORTED, INFINI_ERR_ALIGN = -1, -2, -3, -4
INFINI_ERR_CUDA, INFINI_ERR_TIMEOUT, INFINI_ERR_WORKSPACE, INFINI_ERR_ALIAS, INFINI_ERR_SIZE = -5, -6, -7, -8, -9
INFINI_ERR_SCRATCH = -10
INFINI_ERR_BOUNDS = -11
INFINI_ERR_OFFSETS = -12
INFINI_NOALLOC_SCRATCH_BYTES = 64 << 20
INFINI_PATH_AUTO, INFINI_PATH_SIMT, INFINI_PATH_TC, INFINI_PATH_TC_PAIRED = 0, 1, 2, 3
INFINI_PATH_SPLIT = 4

EXPORTED = ("infini_attn_forward", "infini_attn_workspace_size", "infini_attn_forward_ws",
            "infini_attn_forward_traced", "infini_attn_forward_noalloc",
            "infini_attn_select_path", "infini_attn_launch_count", "infini_attn_device_status",
            "infini_attn_selftest_timeout", "infini_attn_decode_step", "infini_attn_decode_workspace_size",
            "infini_attn_state_ws", "infini_attn_finish_ws", "infini_attn_exscan_parts",
            "infini_attn_backward", "infini_attn_backward_path", "infini_attn_backward_workspace_size",
            "infini_attn_schedule_check",
            "infini_attn_packed_workspace_size", "infini_attn_packed_select_path", "infini_attn_packed_forward",
            "infini_attn_packed_backward_workspace_size", "infini_attn_packed_backward",
            "infini_attn_delta_workspace_size", "infini_attn_delta_forward",
            "infini_attn_delta_backward_workspace_size", "infini_attn_delta_backward", "infini_attn_delta_step",
            "infini_attn_strerror", "infini_attn_version")


class infini_shape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int64), ("H", ctypes.c_int64), ("L", ctypes.c_int64),
                ("d", ctypes.c_int64), ("dtype", ctypes.c_int32)]


class infini_rows(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("stride_t", ctypes.c_int64), ("stride_h", ctypes.c_int64)]


class infini_packed_shape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("n_seq", "Tq", "Tk", "Hq", "Hkv", "d", "max_q", "max_k")] + \
        [("dtype", ctypes.c_int32), ("scale", ctypes.c_float)]


class infini_delta_shape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("n_seq", "T", "Hk", "Hv", "d", "max_len")] + \
        [("dtype", ctypes.c_int32), ("scale", ctypes.c_float)]


_vp, _i64, _sz, _int = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int
_shp = ctypes.POINTER(infini_shape)
_rows, _pshp, _dshp = (ctypes.POINTER(c) for c in (infini_rows, infini_packed_shape, infini_delta_shape))

def _declare(lib):
    """Sets the argument and result types of every entry point on `lib`."""
    lib.infini_attn_forward.argtypes = [_shp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _vp, _vp, _vp, _vp]
    lib.infini_attn_forward.restype = _int
    lib.infini_attn_forward_ws.argtypes = [_shp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _vp, _vp, _vp,
                                            _vp, _sz, _int, _vp]
    lib.infini_attn_forward_ws.restype = _int
    lib.infini_attn_forward_traced.argtypes = [_shp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _vp, _vp, _vp,
                                                _vp, _sz, _int, _vp, _int, _vp]
    lib.infini_attn_forward_traced.restype = _int
    lib.infini_attn_forward_noalloc.argtypes = [_shp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _vp, _vp, _vp, _vp]
    lib.infini_attn_forward_noalloc.restype = _int
    lib.infini_attn_workspace_size.argtypes = [_shp, _i64]
    lib.infini_attn_workspace_size.restype = _sz
    lib.infini_attn_select_path.argtypes = [_shp, _i64]
    lib.infini_attn_select_path.restype = _int
    lib.infini_attn_launch_count.argtypes = [_shp, _i64, _int]
    lib.infini_attn_launch_count.restype = _int
    lib.infini_attn_device_status.argtypes = [_vp]
    lib.infini_attn_device_status.restype = _int
    lib.infini_attn_decode_step.argtypes = [_shp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _vp, _vp, _vp, _vp, _sz, _vp]
    lib.infini_attn_decode_step.restype = _int
    lib.infini_attn_decode_workspace_size.argtypes = [_shp]
    lib.infini_attn_decode_workspace_size.restype = _sz
    lib.infini_attn_state_ws.argtypes = [_shp, _vp, _vp, _i64, _vp, _vp, _vp, _sz, _int, _vp]
    lib.infini_attn_state_ws.restype = _int
    lib.infini_attn_finish_ws.argtypes = [_shp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _vp, _vp, _vp, _vp, _sz, _int, _vp]
    lib.infini_attn_finish_ws.restype = _int
    lib.infini_attn_exscan_parts.argtypes = [_i64, _i64, _int, _int, _vp, _vp, _vp, _vp, _vp, _vp, _vp]
    lib.infini_attn_exscan_parts.restype = _int
    lib.infini_attn_backward_workspace_size.argtypes = [_shp, _i64]
    lib.infini_attn_backward_workspace_size.restype = _sz
    lib.infini_attn_backward.argtypes = [_shp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                          _vp, _vp, _vp, _sz, _vp]
    lib.infini_attn_backward.restype = _int
    lib.infini_attn_backward_path.argtypes = [_shp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _vp,
                                               _vp, _vp, _vp, _vp, _sz, _int, _vp]
    lib.infini_attn_backward_path.restype = _int
    lib.infini_attn_selftest_timeout.argtypes = [ctypes.c_uint64, _vp]
    lib.infini_attn_selftest_timeout.restype = _int
    lib.infini_attn_schedule_check.argtypes = [_i64, _int, _int, ctypes.POINTER(ctypes.c_double)]
    lib.infini_attn_schedule_check.restype = _int
    for name, shape, extra in (("packed", _pshp, [_int]), ("packed_backward", _pshp, []), ("delta", _dshp, [_int]),
                               ("delta_backward", _dshp, [_int])):
        fn = getattr(lib, "infini_attn_%s_workspace_size" % name)
        fn.argtypes, fn.restype = [shape] + extra, _sz
    tail = [_vp, _sz, _int, _vp]  # workspace, its bytes, path, stream
    lib.infini_attn_packed_select_path.argtypes = [_pshp]
    lib.infini_attn_packed_forward.argtypes = [_pshp] + [_rows] * 3 + [_vp] * 4 + [_rows, _vp] + tail
    lib.infini_attn_packed_backward.argtypes = [_pshp] + [_rows] * 4 + [_vp, _rows] + [_vp] * 4 + [_rows] * 3 + tail
    lib.infini_attn_delta_forward.argtypes = [_dshp] + [_rows] * 5 + [_vp] * 3 + [_rows, _vp] + tail
    lib.infini_attn_delta_backward.argtypes = [_dshp] + [_rows] * 5 + [_vp] * 3 + [_rows, _vp] + [_rows] * 5 + [_vp] + tail
    lib.infini_attn_delta_step.argtypes = [_dshp] + [_rows] * 5 + [_vp, _rows, _vp, _vp]
    for name in ("packed_select_path", "packed_forward", "packed_backward", "delta_forward", "delta_backward",
                 "delta_step"):
        getattr(lib, "infini_attn_" + name).restype = _int
    lib.infini_attn_strerror.argtypes = [_int]
    lib.infini_attn_strerror.restype = ctypes.c_char_p
    lib.infini_attn_version.argtypes = []
    lib.infini_attn_version.restype = _int
    return lib


_lib = _declare(_lib)


def open_library(path: str):
    """Another build of the same C ABI (the tracing or the debug build of
    compressive_memory_segment_b200.build), with its entry points declared;
    call them with plain pointers, like the functions below."""
    return _declare(ctypes.CDLL(path))


def _ptr(x) -> Optional[int]:
    """A tensor's data pointer, an int, or None (NULL)."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def make_shape(B: int, H: int, L: int, d: int, dtype: int) -> infini_shape:
    return infini_shape(B, H, L, d, dtype)


def infini_attn_strerror(code: int) -> str:
    return _lib.infini_attn_strerror(code).decode()


def infini_attn_version() -> int:
    return _lib.infini_attn_version()


def infini_attn_workspace_size(shape: infini_shape, seg_len: int) -> int:
    return _lib.infini_attn_workspace_size(ctypes.byref(shape), seg_len)


def infini_attn_select_path(shape: infini_shape, seg_len: int) -> int:
    return _lib.infini_attn_select_path(ctypes.byref(shape), seg_len)


def infini_attn_launch_count(shape: infini_shape, seg_len: int, path: int = INFINI_PATH_AUTO) -> int:
    return _lib.infini_attn_launch_count(ctypes.byref(shape), seg_len, path)


def infini_attn_device_status(stream=None) -> int:
    return _lib.infini_attn_device_status(_stream(stream))


def infini_attn_schedule_check(n_seg: int, n_qt: int, grid: int):
    """(return code, busiest CTA's key tiles over the mean) of the attention
    kernel's unit schedule, run on the host."""
    ratio = ctypes.c_double(0.0)
    rc = _lib.infini_attn_schedule_check(int(n_seg), int(n_qt), int(grid), ctypes.byref(ratio))
    return rc, ratio.value


def infini_attn_selftest_timeout(limit_ns: int, stream=None) -> int:
    return _lib.infini_attn_selftest_timeout(int(limit_ns), _stream(stream))


def infini_attn_forward(shape, q, k, v, beta, M_in, z_in, seg_len, out, M_out, z_out, stream=None) -> int:
    return _lib.infini_attn_forward(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(beta),
                                    _ptr(M_in), _ptr(z_in), seg_len, _ptr(out), _ptr(M_out),
                                    _ptr(z_out), _stream(stream))


def infini_attn_forward_ws(shape, q, k, v, beta, M_in, z_in, seg_len, out, M_out, z_out,
                           workspace, workspace_bytes, path=INFINI_PATH_AUTO, stream=None) -> int:
    return _lib.infini_attn_forward_ws(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(beta),
                                       _ptr(M_in), _ptr(z_in), seg_len, _ptr(out), _ptr(M_out),
                                       _ptr(z_out), _ptr(workspace), workspace_bytes, path,
                                       _stream(stream))


def infini_attn_forward_traced(shape, q, k, v, beta, M_in, z_in, seg_len, out, M_out, z_out,
                               workspace, workspace_bytes, path, events, stream=None) -> int:
    """events: a sequence of torch.cuda.Event (already recorded once, so the
    handle exists) or raw cudaEvent_t ints, launch_count + 1 of them."""
    n = len(events)
    arr = (ctypes.c_void_p * n)(*[e if isinstance(e, int) else e.cuda_event for e in events])
    return _lib.infini_attn_forward_traced(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(beta),
                                           _ptr(M_in), _ptr(z_in), seg_len, _ptr(out), _ptr(M_out),
                                           _ptr(z_out), _ptr(workspace), workspace_bytes, path,
                                           arr, n, _stream(stream))


def infini_attn_forward_noalloc(shape, q, k, v, beta, M_in, z_in, seg_len, out, M_out, z_out,
                                stream=None) -> int:
    """The allocation-free entry point: scratch comes from the library's
    built-in buffer (see the header for the size limit and the rules on
    overlapping calls)."""
    return _lib.infini_attn_forward_noalloc(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(beta),
                                            _ptr(M_in), _ptr(z_in), seg_len, _ptr(out), _ptr(M_out),
                                            _ptr(z_out), _stream(stream))


def infini_attn_decode_workspace_size(shape) -> int:
    return _lib.infini_attn_decode_workspace_size(ctypes.byref(shape))


def infini_attn_decode_step(shape, q, k, v, beta, k_cache, v_cache, pos, M, z, out, workspace, ws_bytes,
                            stream=None) -> int:
    return _lib.infini_attn_decode_step(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(beta),
                                        _ptr(k_cache), _ptr(v_cache), int(pos), _ptr(M), _ptr(z), _ptr(out),
                                        _ptr(workspace), ws_bytes, _stream(stream))


def infini_attn_state_ws(shape, k, v, seg_len, M_tot, z_tot, workspace, workspace_bytes,
                         path=INFINI_PATH_AUTO, stream=None) -> int:
    return _lib.infini_attn_state_ws(ctypes.byref(shape), _ptr(k), _ptr(v), seg_len, _ptr(M_tot), _ptr(z_tot),
                                     _ptr(workspace), workspace_bytes, path, _stream(stream))


def infini_attn_finish_ws(shape, q, k, v, beta, M_in, z_in, seg_len, out, M_out, z_out, workspace,
                          workspace_bytes, path=INFINI_PATH_AUTO, stream=None) -> int:
    return _lib.infini_attn_finish_ws(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(M_in),
                                      _ptr(z_in), seg_len, _ptr(out), _ptr(M_out), _ptr(z_out), _ptr(workspace),
                                      workspace_bytes, path, _stream(stream))


def infini_attn_exscan_parts(n_M, n_z, n_parts, part, totals_M, totals_z, M_in, z_in, off_M, off_z,
                             stream=None) -> int:
    return _lib.infini_attn_exscan_parts(n_M, n_z, n_parts, part, _ptr(totals_M), _ptr(totals_z), _ptr(M_in),
                                         _ptr(z_in), _ptr(off_M), _ptr(off_z), _stream(stream))


def infini_attn_backward_workspace_size(shape, seg_len) -> int:
    return _lib.infini_attn_backward_workspace_size(ctypes.byref(shape), seg_len)


def infini_attn_backward(shape, q, k, v, beta, M_in, z_in, seg_len, dout, dM_out, dz_out, dq, dk, dv, dbeta,
                         dM_in, dz_in, workspace, workspace_bytes, stream=None) -> int:
    return _lib.infini_attn_backward(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(M_in),
                                     _ptr(z_in), seg_len, _ptr(dout), _ptr(dM_out), _ptr(dz_out), _ptr(dq),
                                     _ptr(dk), _ptr(dv), _ptr(dbeta), _ptr(dM_in), _ptr(dz_in), _ptr(workspace),
                                     workspace_bytes, _stream(stream))


def infini_attn_backward_path(shape, q, k, v, beta, M_in, z_in, seg_len, dout, dM_out, dz_out, dq, dk, dv, dbeta,
                              dM_in, dz_in, workspace, workspace_bytes, path, stream=None) -> int:
    return _lib.infini_attn_backward_path(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(M_in),
                                          _ptr(z_in), seg_len, _ptr(dout), _ptr(dM_out), _ptr(dz_out), _ptr(dq),
                                          _ptr(dk), _ptr(dv), _ptr(dbeta), _ptr(dM_in), _ptr(dz_in),
                                          _ptr(workspace), workspace_bytes, path, _stream(stream))


class InfiniError(RuntimeError):
    def __init__(self, code: int):
        super().__init__("infini_attn error %d: %s" % (code, infini_attn_strerror(code)))
        self.code = code


def check(code: int) -> None:
    if code != INFINI_OK:
        raise InfiniError(code)


def shape_of(q) -> infini_shape:
    import torch
    if q.dim() != 4:
        raise ValueError("q must be [B, H, L, d]")
    dt = {torch.float32: INFINI_F32, torch.bfloat16: INFINI_BF16}.get(q.dtype)
    if dt is None:
        raise TypeError("q, k, v must be float32 or bfloat16")
    B, H, L, d = q.shape
    return infini_shape(B, H, L, d, dt)


def workspace_for(q, seg_len: int):
    """Allocate (torch, on q's device) a workspace for this shape."""
    import torch
    n = infini_attn_workspace_size(shape_of(q), seg_len)
    if n == 0:
        raise InfiniError(INFINI_ERR_SHAPE)
    return torch.empty(n, dtype=torch.uint8, device=q.device)


def forward(q, k, v, beta, seg_len: int, M_in=None, z_in=None, out=None, M_out=None, z_out=None,
            workspace=None, path: int = INFINI_PATH_AUTO, stream=None):
    """Run the layer on device tensors q, k, v [B, H, L, d] (fp32 or bf16),
    beta [H] fp32, optional incoming state M_in [B, H, d, d], z_in [B, H, d]
    fp32. Returns (out, M_out, z_out); outputs are allocated when not given."""
    import torch
    shp = shape_of(q)
    B, H, L, d = q.shape
    for t in (q, k, v):
        if not t.is_contiguous():
            raise ValueError("q, k, v must be contiguous")
    if out is None:
        out = torch.empty_like(q)
    if M_out is None:
        M_out = torch.empty((B, H, d, d), dtype=torch.float32, device=q.device)
    if z_out is None:
        z_out = torch.empty((B, H, d), dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = workspace_for(q, seg_len)
    check(infini_attn_forward_ws(shp, q, k, v, beta, M_in, z_in, seg_len, out, M_out, z_out,
                                 workspace, workspace.numel() * workspace.element_size(), path, stream))
    return out, M_out, z_out


def decode_step(q, k, v, beta, k_cache, v_cache, pos: int, M, z, out=None, workspace=None, stream=None):
    """One decode step on device tensors: q, k, v [B, H, d] (this token),
    k_cache, v_cache [B, H, N, d] (rows 0..pos-1 filled; row pos is written),
    M [B, H, d, d] and z [B, H, d] fp32 (updated in place when pos == N - 1).
    Returns out [B, H, d]."""
    import torch
    B, H, N, d = k_cache.shape
    dt = {torch.float32: INFINI_F32, torch.bfloat16: INFINI_BF16}.get(q.dtype)
    if dt is None:
        raise TypeError("q, k, v must be float32 or bfloat16")
    shp = infini_shape(B, H, N, d, dt)
    if out is None:
        out = torch.empty_like(q)
    if workspace is None:
        workspace = torch.empty(infini_attn_decode_workspace_size(shp), dtype=torch.uint8, device=q.device)
    nbytes = workspace.numel() * workspace.element_size()
    check(infini_attn_decode_step(shp, q, k, v, beta, k_cache, v_cache, pos, M, z, out, workspace, nbytes, stream))
    return out


def backward(q, k, v, beta, seg_len: int, dout, M_in=None, z_in=None, dM_out=None, dz_out=None, workspace=None,
             stream=None, path: int = 0):
    """Gradients of the forward on device tensors. Returns (dq, dk, dv, dbeta,
    dM_in, dz_in), all fp32; dq, dk, dv have q's shape. path: INFINI_PATH_AUTO
    (0), _SIMT or _TC."""
    import torch
    shp = shape_of(q)
    B, H, L, d = q.shape
    f32 = dict(dtype=torch.float32, device=q.device)
    dq, dk, dv = (torch.empty((B, H, L, d), **f32) for _ in range(3))
    dbeta = torch.empty((H,), **f32)
    dM_in = torch.empty((B, H, d, d), **f32)
    dz_in = torch.empty((B, H, d), **f32)
    if workspace is None:
        workspace = torch.empty(infini_attn_backward_workspace_size(shp, seg_len), dtype=torch.uint8,
                                device=q.device)
    check(infini_attn_backward_path(shp, q, k, v, beta, M_in, z_in, seg_len, dout, dM_out, dz_out, dq, dk, dv, dbeta,
                                    dM_in, dz_in, workspace, workspace.numel() * workspace.element_size(), path,
                                    stream))
    return dq, dk, dv, dbeta, dM_in, dz_in


# ------------------------------------------------------- packed sequences
# Tensors are [T, H, d] (any strides that the library takes: the last
# dimension contiguous, the others positive multiples of 16 bytes), so slices
# of a fused projection and transposed [H, T, d] buffers are passed as they are.
# The small calls take microseconds on the device, so marshalling is kept lean:
# shapes and rows go over as packed bytes of their C structs.
_lean = ctypes.CDLL(LIB_PATH)
_pack_rows, _pack_packed, _pack_delta = (struct.Struct(f).pack for f in ("=3q", "=8qif", "=6qif"))
for _name in ("packed_workspace_size", "packed_backward_workspace_size", "delta_workspace_size",
              "delta_backward_workspace_size", "packed_forward", "packed_backward", "delta_forward", "delta_backward",
              "delta_step"):
    _fn, _typed = getattr(_lean, "infini_attn_" + _name), getattr(_lib, "infini_attn_" + _name)
    _fn.restype = _typed.restype
    _fn.argtypes = [_vp if t in (_rows, _pshp, _dshp) else t for t in _typed.argtypes]


def _dtype_of(q) -> int:
    import torch
    if q.dtype is torch.bfloat16:
        return INFINI_BF16
    if q.dtype is torch.float32:
        return INFINI_F32
    raise TypeError("q, k, v must be float32 or bfloat16")


def _rows_arg(name, x, dtype, dev, shape):
    """The bytes of infini_rows for a [T, H, d] (or [T, H]) tensor of q's dtype on q's device."""
    if x.shape != shape:
        raise ValueError("%s must be %s, got %s" % (name, list(shape), list(x.shape)))
    if x.dtype is not dtype:
        raise TypeError("%s must be %s like q" % (name, dtype))
    if x.get_device() != dev:
        raise ValueError("%s is on %s, not on q's device" % (name, x.device))
    st = x.stride()
    if len(st) == 3 and st[2] != 1:
        raise ValueError("the last dimension of %s must be contiguous" % name)
    return _pack_rows(x.data_ptr(), st[0], st[1])


def _flat_arg(name, x, dtype, dev, shape):
    """Pointer of a contiguous tensor, or None."""
    if x is None:
        return None
    if x.dtype is not dtype:
        raise TypeError("%s must be %s" % (name, dtype))
    if x.shape != shape:
        raise ValueError("%s must be %s, got %s" % (name, list(shape), list(x.shape)))
    if x.get_device() != dev:
        raise ValueError("%s is on %s, not on q's device" % (name, x.device))
    if not x.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return x.data_ptr()


def _sequences(name, off):
    if off.dim() != 1 or off.shape[0] < 1:
        raise ValueError("%s must be [n_seq + 1]" % name)
    return off.shape[0] - 1


def _device_of(x):
    return x.device


def _streamed(fn):
    """Adds the argument `stream` (a torch stream or a raw handle of q's device;
    None: the current one). The call, and what it allocates, belongs to that
    stream."""
    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        if stream is None or not (args or "q" in kw):
            return fn(*args, **kw)
        import torch
        dev = _device_of(args[0] if args else kw["q"])
        if dev.type != "cuda":
            raise ValueError("q must be on a CUDA device")
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=dev)
        elif stream.device != dev:
            raise ValueError("the stream is on %s, not on q's device" % stream.device)
        with torch.cuda.stream(stream):
            return fn(*args, **kw)
    return call


def _call(fn, dev, *args):
    """fn(*args, stream) on the current stream of device `dev`, with that device current."""
    import torch
    if dev < 0:
        raise ValueError("q must be on a CUDA device")
    stream = torch._C._cuda_getCurrentRawStream(dev)
    if torch._C._cuda_getDevice() == dev:
        rc = fn(*args, stream)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, stream)
    if rc != INFINI_OK:
        raise InfiniError(rc)


def _workspace(workspace, need, q, dev):
    """(tensor to keep, pointer, bytes) of the scratch memory; none is needed up to 256 bytes."""
    if workspace is None:
        if need <= 256:
            return None, None, 0
        import torch
        workspace = q.new_empty(need, dtype=torch.uint8)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous and on q's device")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def packed_shape(q, k, q_off, max_q=None, max_k=None, scale=None) -> infini_packed_shape:
    """The shape of a packed attention call on q [Tq, Hq, d], k [Tk, Hkv, d]
    (for the workspace size functions)."""
    return infini_packed_shape.from_buffer_copy(_packed_bytes(q, k, _sequences("q_off", q_off), max_q, max_k, scale))


def _packed_bytes(q, k, n, max_q, max_k, scale):
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q, k, v must be [T, H, d]")
    (Tq, Hq, d), (Tk, Hkv, _) = q.shape, k.shape
    return _pack_packed(n, Tq, Tk, Hq, Hkv, d, Tq if max_q is None else max_q, Tk if max_k is None else max_k,
                        _dtype_of(q), d ** -0.5 if scale is None else scale)


@_streamed
def packed_forward(q, k, v, q_off, k_off=None, q_len=None, k_len=None, max_q=None, max_k=None, scale=None, out=None,
                   lse=None, workspace=None, path: int = INFINI_PATH_AUTO):
    """Causal softmax attention over packed sequences with grouped heads: q
    [Tq, Hq, d], k, v [Tk, Hkv, d] (fp32 or bf16), Hq a multiple of Hkv.
    Sequence s has the query rows q_off[s]..q_off[s + 1] and the keys of k_off
    (default q_off, k_len then q_len), int32 on the device; q_len, k_len shorten
    them (a padded batch, a cache). The last query sees every key. max_q, max_k:
    the longest sequence's queries and keys where the caller knows them (give
    max_q = 1 for a step against a cache). Returns (out [Tq, Hq, d], lse
    [Hq, Tq] fp32); both are allocated when not given (rows of no sequence are
    left as they are: unset in a new tensor)."""
    import torch
    n = _sequences("q_off", q_off)
    shp = _packed_bytes(q, k, n, max_q, max_k, scale)
    dt, dev, i32 = q.dtype, q.get_device(), torch.int32
    qs, ks = q.shape, k.shape
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = q.new_empty((qs[1], qs[0]), dtype=torch.float32)
    at = _flat_arg("q_off", q_off, i32, dev, (n + 1,))
    if k_off is None:
        at_k, k_len = at, q_len if k_len is None else k_len
    else:
        at_k = _flat_arg("k_off", k_off, i32, dev, (n + 1,))
    _keep, ws, nbytes = _workspace(workspace, _lean.infini_attn_packed_workspace_size(shp, path), q, dev)
    _call(_lean.infini_attn_packed_forward, dev, shp, _rows_arg("q", q, dt, dev, qs),
          _rows_arg("k", k, dt, dev, (ks[0], ks[1], qs[2])), _rows_arg("v", v, dt, dev, ks), at, at_k,
          _flat_arg("q_len", q_len, i32, dev, (n,)), _flat_arg("k_len", k_len, i32, dev, (n,)),
          _rows_arg("out", out, dt, dev, qs), _flat_arg("lse", lse, torch.float32, dev, (qs[1], qs[0])), ws, nbytes, path)
    return out, lse


@_streamed
def packed_backward(q, k, v, out, lse, dout, q_off, k_off=None, q_len=None, k_len=None, max_q=None, max_k=None,
                    scale=None, dq=None, dk=None, dv=None, workspace=None, path: int = INFINI_PATH_AUTO):
    """Gradients of packed_forward for dout [Tq, Hq, d], from its out and lse.
    Returns (dq, dk, dv) in q's dtype, allocated when not given (rows of no
    sequence are left as they are: unset in a new tensor)."""
    import torch
    n = _sequences("q_off", q_off)
    shp = _packed_bytes(q, k, n, max_q, max_k, scale)
    dt, dev, i32 = q.dtype, q.get_device(), torch.int32
    qs, ks = q.shape, k.shape
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    at = _flat_arg("q_off", q_off, i32, dev, (n + 1,))
    if k_off is None:
        at_k, k_len = at, q_len if k_len is None else k_len
    else:
        at_k = _flat_arg("k_off", k_off, i32, dev, (n + 1,))
    _keep, ws, nbytes = _workspace(workspace, _lean.infini_attn_packed_backward_workspace_size(shp), q, dev)
    _call(_lean.infini_attn_packed_backward, dev, shp, _rows_arg("q", q, dt, dev, qs),
          _rows_arg("k", k, dt, dev, (ks[0], ks[1], qs[2])), _rows_arg("v", v, dt, dev, ks),
          _rows_arg("out", out, dt, dev, qs), _flat_arg("lse", lse, torch.float32, dev, (qs[1], qs[0])),
          _rows_arg("dout", dout, dt, dev, qs), at, at_k, _flat_arg("q_len", q_len, i32, dev, (n,)),
          _flat_arg("k_len", k_len, i32, dev, (n,)), _rows_arg("dq", dq, dt, dev, qs), _rows_arg("dk", dk, dt, dev, ks),
          _rows_arg("dv", dv, dt, dev, ks), ws, nbytes, path)
    return dq, dk, dv


def delta_shape(q, v, n_seq, max_len=None, scale=None) -> infini_delta_shape:
    """The shape of a delta-rule call on q [T, Hk, d], v [T, Hv, d] (for the
    workspace size functions)."""
    return infini_delta_shape.from_buffer_copy(_delta_bytes(q, v, n_seq, max_len, scale))


def _delta_bytes(q, v, n, max_len, scale):
    if q.dim() != 3 or v.dim() != 3:
        raise ValueError("q, k, v must be [T, H, d]")
    T, Hk, d = q.shape
    return _pack_delta(n, T, Hk, v.shape[1], d, T if max_len is None else max_len, _dtype_of(q),
                       d ** -0.5 if scale is None else scale)


def _delta_rows(q, k, v, g, beta, dt, dev):
    qs, vs = q.shape, (q.shape[0], v.shape[1], q.shape[2])
    return (_rows_arg("q", q, dt, dev, qs), _rows_arg("k", k, dt, dev, qs), _rows_arg("v", v, dt, dev, vs),
            _rows_arg("g", g, dt, dev, vs[:2]), _rows_arg("beta", beta, dt, dev, vs[:2]))


@_streamed
def delta_forward(q, k, v, g, beta, off, seq_len=None, S_in=None, scale=None, max_len=None, out=None, S_out=None,
                  workspace=None, path: int = INFINI_PATH_AUTO):
    """The gated delta rule over packed sequences: q, k [T, Hk, d], v [T, Hv, d],
    g (log decay), beta [T, Hv] in one dtype (fp32 or bf16), Hv a multiple of
    Hk; sequence s has the rows off[s]..off[s + 1] (int32 on the device), of
    which seq_len[s] count. S_in [n_seq, Hv, d, d] fp32 (None: zero). scale:
    default d ** -0.5. max_len: the longest sequence where the caller knows it.
    Returns (out [T, Hv, d], S_out), allocated when not given; S_out may be S_in
    itself."""
    import torch
    n = _sequences("off", off)
    shp = _delta_bytes(q, v, n, max_len, scale)
    dt, dev, i32, f32 = q.dtype, q.get_device(), torch.int32, torch.float32
    vs = v.shape
    state = (n, vs[1], vs[2], vs[2])
    if out is None:
        out = torch.empty_like(v)
    if S_out is None:
        S_out = q.new_empty(state, dtype=f32)
    _keep, ws, nbytes = _workspace(workspace, _lean.infini_attn_delta_workspace_size(shp, path), q, dev)
    _call(_lean.infini_attn_delta_forward, dev, shp, *_delta_rows(q, k, v, g, beta, dt, dev),
          _flat_arg("off", off, i32, dev, (n + 1,)), _flat_arg("seq_len", seq_len, i32, dev, (n,)),
          _flat_arg("S_in", S_in, f32, dev, state), _rows_arg("out", out, dt, dev, vs),
          _flat_arg("S_out", S_out, f32, dev, state), ws, nbytes, path)
    return out, S_out


@_streamed
def delta_backward(q, k, v, g, beta, off, dout, seq_len=None, S_in=None, dS_out=None, scale=None, max_len=None,
                   dq=None, dk=None, dv=None, dg=None, dbeta=None, dS_in=None, workspace=None,
                   path: int = INFINI_PATH_AUTO):
    """Gradients of delta_forward for dout [T, Hv, d] and dS_out (None: zero).
    Returns (dq, dk, dv, dg, dbeta, dS_in), the first five in q's dtype, dS_in
    fp32, allocated when not given (rows of no sequence are left as they are:
    unset in a new tensor)."""
    import torch
    n = _sequences("off", off)
    shp = _delta_bytes(q, v, n, max_len, scale)
    dt, dev, i32, f32 = q.dtype, q.get_device(), torch.int32, torch.float32
    qs, vs = q.shape, v.shape
    state = (n, vs[1], vs[2], vs[2])
    new = lambda x, like: torch.empty_like(like) if x is None else x  # noqa: E731
    dq, dk, dv, dg, dbeta = new(dq, q), new(dk, k), new(dv, v), new(dg, g), new(dbeta, beta)
    dS_in = q.new_empty(state, dtype=f32) if dS_in is None else dS_in
    _keep, ws, nbytes = _workspace(workspace, _lean.infini_attn_delta_backward_workspace_size(shp, path), q, dev)
    _call(_lean.infini_attn_delta_backward, dev, shp, *_delta_rows(q, k, v, g, beta, dt, dev),
          _flat_arg("off", off, i32, dev, (n + 1,)), _flat_arg("seq_len", seq_len, i32, dev, (n,)),
          _flat_arg("S_in", S_in, f32, dev, state), _rows_arg("dout", dout, dt, dev, vs),
          _flat_arg("dS_out", dS_out, f32, dev, state), _rows_arg("dq", dq, dt, dev, qs), _rows_arg("dk", dk, dt, dev, qs),
          _rows_arg("dv", dv, dt, dev, vs), _rows_arg("dg", dg, dt, dev, vs[:2]),
          _rows_arg("dbeta", dbeta, dt, dev, vs[:2]), _flat_arg("dS_in", dS_in, f32, dev, state), ws, nbytes, path)
    return dq, dk, dv, dg, dbeta, dS_in


@_streamed
def delta_step(q, k, v, g, beta, S, S_out=None, scale=None, out=None):
    """One token for each of B states: q, k [B, Hk, d], v [B, Hv, d], g, beta
    [B, Hv], S [B, Hv, d, d] fp32, updated in place unless S_out is given.
    Returns out [B, Hv, d]."""
    import torch
    shp = _delta_bytes(q, v, 0, 0, scale)
    dt, dev, f32 = q.dtype, q.get_device(), torch.float32
    vs = v.shape
    state = (vs[0], vs[1], vs[2], vs[2])
    if out is None:
        out = torch.empty_like(v)
    S_ptr = _flat_arg("S", S, f32, dev, state)
    to = S_ptr if S_out is None else _flat_arg("S_out", S_out, f32, dev, state)
    _call(_lean.infini_attn_delta_step, dev, shp, *_delta_rows(q, k, v, g, beta, dt, dev), S_ptr,
          _rows_arg("out", out, dt, dev, vs), to)
    return out
