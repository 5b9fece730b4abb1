"""ctypes binding of the lapmix operators (include/lapmix.h): argument marshalling only.

The gated linear recurrence (``lapmix_scan_*``) and the root-mean-square norm
with the residual's addition (``lapmix_norm_*``), in the manner of the attention's
binding: functions carry the names of the C entry points, outputs are given by the
caller, tensors are device tensors of the current device, and a negative status
raises ``LapnysError``.  [B, H, N, d] tensors may be views with any strides as long
as channels are contiguous (a permuted [B, N, H, d] tensor, a slice of a projection):
the binding passes their strides.  Plain integers are raw device pointers, with the
strides that the params hold.
"""

from __future__ import annotations

import ctypes

import torch

from .lapnys import LAPNYS_BF16, LAPNYS_F32, _check, _lib, _stream as _given_stream, _ws

LAPMIX_E4M3 = 2
LAPMIX_GATE_LOG = 1
LAPMIX_COUPLED = 2
LAPMIX_SCAN_TILE = 128

_SIZES = {LAPNYS_F32: 4, LAPNYS_BF16: 2, LAPMIX_E4M3: 1}
_INDEX = (torch.int32,)
# Tensor types by element size: the storage types, or their bit patterns.
_TYPES = {4: (torch.float32,), 2: (torch.bfloat16, torch.int16, torch.uint16),
          1: (torch.float8_e4m3fn, torch.uint8, torch.int8)}
_NAMES = {"f32": LAPNYS_F32, "bf16": LAPNYS_BF16, "e4m3": LAPMIX_E4M3}
_stride = ctypes.c_int64 * 3


class lapmix_scan_params(ctypes.Structure):
    """Mirror of the C struct."""

    _fields_ = [("B", ctypes.c_int32), ("H", ctypes.c_int32), ("N", ctypes.c_int32), ("d", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("flags", ctypes.c_uint32),
                ("x_stride", _stride), ("g_stride", _stride), ("y_stride", _stride)]


class lapmix_norm_params(ctypes.Structure):
    """Mirror of the C struct."""

    _fields_ = [("B", ctypes.c_int32), ("H", ctypes.c_int32), ("N", ctypes.c_int32), ("d", ctypes.c_int32),
                ("x_dtype", ctypes.c_int32), ("r_dtype", ctypes.c_int32), ("y_dtype", ctypes.c_int32),
                ("group", ctypes.c_int32), ("eps", ctypes.c_float), ("reserved", ctypes.c_int32),
                ("x_stride", _stride)]


def _declare():
    vp, i32, size = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    S, M = ctypes.POINTER(lapmix_scan_params), ctypes.POINTER(lapmix_norm_params)
    out = ctypes.POINTER(size)
    for name, args in {
        "lapmix_scan_workspace_size": [S, out],
        "lapmix_scan_states_size": [S, out],
        "lapmix_scan_forward_ws": [vp, vp, vp, vp, vp, vp, vp, S, vp, size, vp],
        "lapmix_scan_backward_ws": [vp, vp, vp, vp, vp, vp, vp, vp, vp, S, vp, size, vp],
        "lapmix_scan_step": [vp, vp, vp, vp, vp, i32, vp, S, vp],
        "lapmix_norm_forward": [vp, vp, vp, vp, vp, vp, M, vp],
        "lapmix_norm_workspace_size": [M, out],
        "lapmix_norm_backward_ws": [vp, vp, vp, vp, vp, vp, vp, M, vp, size, vp],
    }.items():
        f = getattr(_lib, name)
        f.argtypes = args
        f.restype = ctypes.c_int


_declare()


def make_scan_params(*, B, H, N, d, dtype="f32", gate="sigmoid", coupled=False) -> lapmix_scan_params:
    """Build a lapmix_scan_params; ``dtype`` is "f32"/"bf16" or the enum value; ``gate`` is "sigmoid"
    (f = sigmoid(g)) or "log" (f = exp(min(g, 0)), LAPMIX_GATE_LOG); ``coupled`` sets
    LAPMIX_COUPLED (the input enters as (1 - f) x)."""
    if gate not in ("sigmoid", "log"):
        raise ValueError(f"unknown gate {gate!r}")
    flags = (LAPMIX_GATE_LOG if gate == "log" else 0) | (LAPMIX_COUPLED if coupled else 0)
    return lapmix_scan_params(B, H, N, d, _NAMES.get(dtype, dtype), flags)


def make_norm_params(*, B, H, N, d, x_dtype="f32", r_dtype="f32", y_dtype="f32", eps=1e-6,
                     group=0) -> lapmix_norm_params:
    """Build a lapmix_norm_params for B * N rows of H * d columns; types are "f32"/"bf16" (``y_dtype``
    also "e4m3") or enum values; ``group`` is the columns to a scale (0: one scale a row)."""
    return lapmix_norm_params(B, H, N, d, _NAMES.get(x_dtype, x_dtype), _NAMES.get(r_dtype, r_dtype),
                              _NAMES.get(y_dtype, y_dtype), group, eps, 0)


# Decoding steps are a few microseconds long on the GPU, so the checks of a call go by
# the shortest ways to a tensor's facts and ask for the current device once (``dev``).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _current():
    """Index of the current device; without a GPU, where every tensor is refused as a host tensor, -1."""
    return torch.cuda.current_device() if torch.cuda.device_count() else -1


def _stream(stream, dev):
    return _raw_stream(dev) if stream is None and dev >= 0 else _given_stream(stream)


def _device_ptr(t, dev):
    if t.get_device() != dev or not t.is_cuda:
        if not t.is_cuda:
            raise ValueError("tensor arguments must be device tensors (got a tensor on the host)")
        raise ValueError(f"tensor on {t.device}, but the current device is cuda:{dev}")
    return t.data_ptr()


def _flat(name, t, size, count, dev, types=None):
    """Pointer of a dense tensor argument that holds at least ``count`` elements of ``size`` bytes."""
    if t is None or isinstance(t, int):
        return t
    if t.dtype not in (types or _TYPES.get(size, ())) or t.numel() < count:
        raise ValueError(f"{name}: expected at least {count} elements of {size} bytes, "
                         f"got {t.numel()} of {t.element_size()} ({t.dtype})")
    if not t.is_contiguous():
        raise ValueError("tensor arguments must be contiguous")
    return _device_ptr(t, dev)


def _heads(name, t, size, shape, dev):
    """(pointer, strides) of a [B, H, N, d] tensor argument; strides None for a raw pointer."""
    if t is None or isinstance(t, int):
        return t, None
    if t.dtype not in _TYPES.get(size, ()) or t.shape != shape:
        raise ValueError(f"{name}: expected {list(shape)} of {size} bytes, "
                         f"got {list(t.shape)} of {t.element_size()} ({t.dtype})")
    ptr = _device_ptr(t, dev)
    b, h, n, c = t.stride()
    B, H, N, d = shape
    if c != 1 and d != 1:
        raise ValueError(f"{name}: channels must be contiguous (stride {c})")
    # Strides of dimensions of size 1 do not matter; all zero would mean a dense tensor.
    st = (b if B > 1 else 0, h if H > 1 else 0, n if N > 1 else 0)
    if st == (0, 0, 0) and B * H * N > 1:
        raise ValueError(f"{name}: one row repeated for every token is not supported")
    return ptr, st


def _agree(name, st, other, of):
    if st is not None and of is not None and st != of:
        raise ValueError(f"{name}: expected the strides of {other}, {of}, got {st}")


def lapmix_scan_workspace_size(params: lapmix_scan_params) -> int:
    n = ctypes.c_size_t(0)
    _check(_lib.lapmix_scan_workspace_size(ctypes.byref(params), ctypes.byref(n)), "lapmix_scan_workspace_size")
    return n.value


def lapmix_scan_states_size(params: lapmix_scan_params) -> int:
    n = ctypes.c_size_t(0)
    _check(_lib.lapmix_scan_states_size(ctypes.byref(params), ctypes.byref(n)), "lapmix_scan_states_size")
    return n.value


def _tiles(N):
    return -(-N // LAPMIX_SCAN_TILE)


def _scan_shape(p):
    """[B, H, N, d], element size and columns of a recurrence, and the current device."""
    B, H, N, d = p.B, p.H, p.N, p.d
    return (B, H, N, d), _SIZES.get(p.dtype, 0), B * H * d, _current()


def _norm_shape(p):
    """[B, H, N, d], row width, elements and the stream's element size of a norm, and the current device."""
    B, H, N, d = p.B, p.H, p.N, p.d
    return (B, H, N, d), H * d, B * N * H * d, _SIZES.get(p.r_dtype, 0), _current()


def _scan_params(params, xs, gs, ys):
    p = lapmix_scan_params.from_buffer_copy(params)
    if xs is not None:
        p.x_stride[:] = xs
    if gs is not None:
        p.g_stride[:] = gs
    if ys is not None:
        p.y_stride[:] = ys
    return ctypes.byref(p)


def lapmix_scan_forward_ws(x, g, y, params: lapmix_scan_params, ws, h0=None, hN=None, states=None, lengths=None,
                           stream=None) -> None:
    """y (and the last state hN, and the states that the backward reads) of h_t = f_t h_{t-1} + i_t x_t."""
    shape, size, cols, dev = _scan_shape(params)
    xp, xs = _heads("x", x, size, shape, dev)
    gp, gs = _heads("g", g, size, shape, dev)
    yp, ys = _heads("y", y, size, shape, dev)
    wp, wn = _ws(ws)
    _check(_lib.lapmix_scan_forward_ws(
        xp, gp, _flat("h0", h0, 4, cols, dev), _flat("lengths", lengths, 4, shape[0], dev, _INDEX), yp,
        _flat("hN", hN, 4, cols, dev), _flat("states", states, 4, cols * _tiles(shape[2]), dev),
        _scan_params(params, xs, gs, ys), wp, wn, _stream(stream, dev)), "lapmix_scan_forward_ws")


def lapmix_scan_backward_ws(x, g, states, dy, dx, dg, params: lapmix_scan_params, ws, dhN=None, dh0=None,
                            lengths=None, stream=None) -> None:
    """Gradients of sum(dy * y) + sum(dhN * hN) into dx, dg and dh0; dx and dg have the strides of x and g."""
    shape, size, cols, dev = _scan_shape(params)
    xp, xs = _heads("x", x, size, shape, dev)
    gp, gs = _heads("g", g, size, shape, dev)
    dyp, ys = _heads("dy", dy, size, shape, dev)
    dxp, dxs = _heads("dx", dx, size, shape, dev)
    dgp, dgs = _heads("dg", dg, size, shape, dev)
    _agree("dx", dxs, "x", xs)
    _agree("dg", dgs, "g", gs)
    wp, wn = _ws(ws)
    _check(_lib.lapmix_scan_backward_ws(
        xp, gp, _flat("states", states, 4, cols * _tiles(shape[2]), dev),
        _flat("lengths", lengths, 4, shape[0], dev, _INDEX), dyp, _flat("dhN", dhN, 4, cols, dev), dxp, dgp,
        _flat("dh0", dh0, 4, cols, dev),
        _scan_params(params, xs, gs, ys), wp, wn, _stream(stream, dev)), "lapmix_scan_backward_ws")


def lapmix_scan_step(x, g, y, h_in, h_out, params: lapmix_scan_params, slots=None, n_slots=None, stream=None) -> None:
    """One token for every sequence: y = h_out[slot] = f h_in[slot] + i x.  ``h_in`` and ``h_out`` are
    float32 [n_slots, H, d] pools (``n_slots`` is taken from h_in's shape unless given)."""
    if n_slots is None:
        if isinstance(h_in, int):
            raise ValueError("n_slots is needed with a raw pool pointer")
        n_slots = h_in.shape[0]
    shape, size, _, dev = _scan_shape(params)
    pool = n_slots * shape[1] * shape[3]
    xp, xs = _heads("x", x, size, shape, dev)
    gp, gs = _heads("g", g, size, shape, dev)
    yp, ys = _heads("y", y, size, shape, dev)
    _check(_lib.lapmix_scan_step(
        xp, gp, _flat("slots", slots, 4, shape[0], dev, _INDEX), _flat("h_in", h_in, 4, pool, dev),
        _flat("h_out", h_out, 4, pool, dev), n_slots, yp, _scan_params(params, xs, gs, ys), _stream(stream, dev)),
        "lapmix_scan_step")


def _norm_params(params, xs):
    if xs is None:
        return ctypes.byref(params)
    p = lapmix_norm_params.from_buffer_copy(params)
    p.x_stride[:] = xs
    return ctypes.byref(p)


def lapmix_norm_forward(x, w, y, params: lapmix_norm_params, r=None, s=None, scale=None, stream=None) -> None:
    """s = x + r and y = s / sqrt(mean(s^2) + eps) * w for every token's row (e4m3: with ``scale``)."""
    p = params
    shape, C, n, rs, dev = _norm_shape(p)
    xp, xs = _heads("x", x, _SIZES.get(p.x_dtype, 0), shape, dev)
    _check(_lib.lapmix_norm_forward(
        xp, _flat("r", r, rs, n, dev), _flat("w", w, 4, C, dev), _flat("s", s, rs, n, dev),
        _flat("y", y, _SIZES.get(p.y_dtype, 0), n, dev), _flat("scale", scale, 4, n // max(p.group or C, 1), dev),
        _norm_params(p, xs), _stream(stream, dev)), "lapmix_norm_forward")


def lapmix_norm_workspace_size(params: lapmix_norm_params) -> int:
    n = ctypes.c_size_t(0)
    _check(_lib.lapmix_norm_workspace_size(ctypes.byref(params), ctypes.byref(n)), "lapmix_norm_workspace_size")
    return n.value


def lapmix_norm_backward_ws(dy, s, w, params: lapmix_norm_params, ws, ds=None, dr=None, dx=None, dw=None,
                            stream=None) -> None:
    """Gradients of sum(dy * y) + sum(ds * s) into dr (the stream's), dx (the branch's) and dw."""
    p = params
    shape, C, n, rs, dev = _norm_shape(p)
    dxp, xs = _heads("dx", dx, _SIZES.get(p.x_dtype, 0), shape, dev)
    wp, wn = _ws(ws)
    _check(_lib.lapmix_norm_backward_ws(
        _flat("dy", dy, _SIZES.get(p.y_dtype, 0), n, dev), _flat("s", s, rs, n, dev), _flat("w", w, 4, C, dev),
        _flat("ds", ds, rs, n, dev), _flat("dr", dr, rs, n, dev), dxp, _flat("dw", dw, 4, C, dev), _norm_params(p, xs),
        wp, wn, _stream(stream, dev)), "lapmix_norm_backward_ws")
