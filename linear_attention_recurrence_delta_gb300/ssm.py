"""State-space layer: Python binding of the operators of ``include/gdn_ssm.h``.

Like the other bindings it only marshals arguments; a tensor given as a view becomes its address and strides, so slices of
a projection's output go in as they are (``xz[:, :D]`` for the convolution, ``bc[:, R:R + N]`` for the scan's vectors).
Rows may be one leading dimension ``[rows, D]`` or ``[B, T, D]`` whose first two collapse into rows; the scan's vectors are
``[rows, G, N]`` (or ``[B, T, G, N]``).  A tensor that is not laid out that way, not of the type that the call reads
(torch.int32 for offsets and slots, torch.float32 for weights, scales and the scan's states, the shape's io for the rest) or
not on the current device raises ValueError; everything else is checked by the library, which returns its status code.

One layer, between its projections (``gdn`` is this package)::

    n = gdn.make_norm(rows, D, "bf16", out="e4m3", group=128)                 # residual stream in, 8-bit rows out
    gdn.check(gdn.gdn_norm_fwd(n, x, res, w, y8, scale, res))
    c = gdn.make_conv(B, T, D, 4, "bf16", rows=rows)
    gdn.check(gdn.gdn_conv_fwd(c, xz[:, :D], taps, bias, cu, s0, u, sT))      # prompts, training
    s = gdn.make_scan(B, T, D, N, 1, "bf16", rows=rows)
    ws = torch.empty(gdn.gdn_scan_workspace_bytes(s, 0), dtype=torch.uint8, device="cuda")
    gdn.check(gdn.gdn_scan_fwd(s, u, dt, xz[:, D:], Bm, Cm, A_log, skip, dt_bias, cu, h0, y, hT, None, ws))
    c1, s1 = gdn.make_conv_step(B, 1, D, 4, slots), gdn.make_scan_step(B, 1, D, N, slots)      # new tokens
    gdn.check(gdn.gdn_conv_step(c1, xz[:, :D], taps, bias, conv_state, slot, None, u))
    gdn.check(gdn.gdn_scan_step(s1, u, dt, xz[:, D:], Bm, Cm, A_log, skip, dt_bias, scan_state, slot, None, y))
"""
from __future__ import annotations

import ctypes

from . import _nbytes, _ptr, _stream, load
from .mla import _IO, _ints, _Shape, _typed, _view, gdn_mla_view_t

GDN_E4M3 = 2


class gdn_norm_t(_Shape):
    _fields_ = _ints("N D io res out group") + [("eps", ctypes.c_float)]


class gdn_conv_t(_Shape):
    _fields_ = _ints("B T D W silu io rows")


class gdn_conv_step_t(_Shape):
    _fields_ = _ints("B T D W silu io slots")


class gdn_scan_t(_Shape):
    _fields_ = _ints("B T D N G softplus io rows")


class gdn_scan_step_t(_Shape):
    _fields_ = _ints("B T D N G softplus io slots")


_OUT = {**_IO, "e4m3": GDN_E4M3}


def make_norm(N, D, io="bf16", res=None, out=None, group=0, eps=1e-6):
    """res: type of the residual stream ("f32", or io as if not given); out: io, or "e4m3" with a scale for each `group`
    values of a row (0: the row)."""
    io = _IO.get(io, io)
    return gdn_norm_t(int(N), int(D), io, io if res is None else _IO.get(res, res), io if out is None else _OUT.get(out, out),
                      int(group), float(eps))


def make_conv(B, T, D, W, io="bf16", silu=True, rows=None):
    """rows: rows of packed tensors (B * T if not given)."""
    return gdn_conv_t(int(B), int(T), int(D), int(W), int(bool(silu)), _IO.get(io, io), int(B * T if rows is None else rows))


def make_conv_step(B, T, D, W, slots, io="bf16", silu=True):
    return gdn_conv_step_t(int(B), int(T), int(D), int(W), int(bool(silu)), _IO.get(io, io), int(slots))


def make_scan(B, T, D, N, G=1, io="bf16", softplus=True, rows=None):
    """rows: rows of packed tensors (B * T if not given)."""
    return gdn_scan_t(int(B), int(T), int(D), int(N), int(G), int(bool(softplus)), _IO.get(io, io),
                      int(B * T if rows is None else rows))


def make_scan_step(B, T, D, N, slots, G=1, io="bf16", softplus=True):
    return gdn_scan_step_t(int(B), int(T), int(D), int(N), int(G), int(bool(softplus)), _IO.get(io, io), int(slots))


_F32 = _I32 = None      # torch's types, from here on known when the library is loaded
_DTYPE = {}             # by gdn_dtype_t (and GDN_E4M3)
_device = _raw_stream = None      # the current device, and its current stream without a Stream object around it


class _Functions(dict):
    """The library's functions by name: loads it when the first one is asked for."""

    def __missing__(self, name):
        self[name] = f = getattr(load(), name)
        return f


_FN = _Functions()


def declare(lib):
    """Signatures of the library's functions (called once, when it is loaded)."""
    global _F32, _I32, _device, _raw_stream
    import torch
    _F32, _I32 = torch.float32, torch.int32
    _DTYPE.update({0: torch.float32, 1: torch.bfloat16, GDN_E4M3: torch.float8_e4m3fn})
    if torch.cuda.is_available():
        _device, _raw_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
    else:
        _device, _raw_stream = lambda: -1, lambda dev: 0
    vp, ll, sz, vw, i = ctypes.c_void_p, ctypes.c_longlong, ctypes.c_size_t, ctypes.POINTER(gdn_mla_view_t), ctypes.c_int
    n, c, cs, s, ss = (ctypes.POINTER(t) for t in (gdn_norm_t, gdn_conv_t, gdn_conv_step_t, gdn_scan_t, gdn_scan_step_t))
    for name, args, res in (
            ("gdn_norm_fwd", [n, vp, ll, vp, ll, vp, vp, ll, vp, vp, ll, vp], i),
            ("gdn_norm_workspace_bytes", [n], sz),
            ("gdn_norm_bwd", [n, vp, ll, vp, vp, ll, vp, ll, vp, ll, vp, ll, vp, vp, sz, vp], i),
            ("gdn_conv_fwd", [c, vw, vp, vp, vp, vp, vw, vp, vp], i),
            ("gdn_conv_workspace_bytes", [c], sz),
            ("gdn_conv_bwd", [c, vw, vp, vp, vp, vp, vw, vp, vw, vp, vp, vp, vp, sz, vp], i),
            ("gdn_conv_step", [cs, vw, vp, vp, vp, vp, vp, vw, vp], i),
            ("gdn_scan_workspace_bytes", [s, i], sz),
            ("gdn_scan_saved_bytes", [s], sz),
            ("gdn_scan_fwd", [s] + [vw] * 5 + [vp] * 5 + [vw, vp, vp, sz, vp, sz, vp], i),
            ("gdn_scan_bwd", [s] + [vw] * 5 + [vp] * 5 + [sz, vw, vp] + [vw] * 5 + [vp] * 5 + [sz, vp], i),
            ("gdn_scan_step", [ss] + [vw] * 5 + [vp] * 6 + [vw, vp], i)):
        f = getattr(lib, name)
        f.argtypes, f.restype = args, res


_ref = ctypes.byref


def _elsewhere(t):
    raise ValueError(f"a tensor on the current CUDA device ({_device()}) is wanted here, not on {t.device}")


def _flat(t, dtype, dev):
    """[rows, D] or [B, T, D] by reference."""
    if t is None:
        return None
    if type(t) is gdn_mla_view_t:
        return _ref(t)
    if t.dtype is not dtype:
        _typed(t, dtype)
    if t.get_device() != dev:
        _elsewhere(t)
    s = t.stride()
    if len(s) == 2 and s[1] == 1 and s[0] % 8 == 0 and s[0] > 0:
        return _ref(gdn_mla_view_t(t.data_ptr(), s[0], s[0]))
    return _ref(_view(t, heads=False))


def _vectors(t, dtype, dev):
    """[rows, G, N] or [B, T, G, N] by reference."""
    if t is None:
        return None
    if type(t) is gdn_mla_view_t:
        return _ref(t)
    if t.dtype is not dtype:
        _typed(t, dtype)
    if t.get_device() != dev:
        _elsewhere(t)
    s = t.stride()
    if len(s) == 3 and s[2] == 1 and s[0] % 8 == 0 and s[0] > 0:
        return _ref(gdn_mla_view_t(t.data_ptr(), s[0], s[1]))
    return _ref(_view(t))


def _rows(t, dtype, dev):
    """[rows, D] as (address, row stride)."""
    if t is None:
        return None, 0
    if type(t) is gdn_mla_view_t:
        return t.p, t.tok
    if t.dtype is not dtype:
        _typed(t, dtype)
    if t.get_device() != dev:
        _elsewhere(t)
    s = t.stride()
    if len(s) == 2 and s[1] == 1 and s[0] % 8 == 0 and s[0] > 0:
        return t.data_ptr(), s[0]
    v = _view(t, heads=False)
    return v.p, v.tok


def _dense(t, dtype, dev):
    """The address of a contiguous tensor."""
    if t is None or type(t) is int:
        return t
    if t.dtype is not dtype:
        _typed(t, dtype)
    if t.get_device() != dev:
        _elsewhere(t)
    if not t.is_contiguous():
        raise ValueError("weights, states, scales, offsets and slots are contiguous")
    return t.data_ptr()


def _area(t, n, dev):
    """A workspace's address and bytes."""
    if t is not None and type(t) is not int and t.get_device() != dev:
        _elsewhere(t)
    return _ptr(t), _nbytes(t) if n is None and t is not None else (n or 0)


def gdn_norm_fwd(shape, x, res, w, y, scale, sum_out, stream=None) -> int:
    """y (and scale, with an 8-bit y) of x + res, which goes to sum_out if given (it may be res itself)."""
    f, d, r, dev = _FN["gdn_norm_fwd"], _DTYPE.get(shape.io), _DTYPE.get(shape.res), _device()
    return f(_ref(shape), *_rows(x, d, dev), *_rows(res, r, dev), _dense(w, _F32, dev),
             *_rows(y, _DTYPE.get(shape.out), dev), _dense(scale, _F32, dev), *_rows(sum_out, r, dev),
             _raw_stream(dev) if stream is None else _stream(stream))


def gdn_norm_workspace_bytes(shape) -> int:
    return load().gdn_norm_workspace_bytes(_ref(shape))


def gdn_norm_bwd(shape, s, w, dy, dsum, dx, dres, dw, ws, ws_bytes=None, stream=None) -> int:
    """From the forward's sum `s`: dx (io), dres (the residual's type) and dw [D] fp32; dsum is the sum's own gradient."""
    f, d, r, dev = _FN["gdn_norm_bwd"], _DTYPE.get(shape.io), _DTYPE.get(shape.res), _device()
    return f(_ref(shape), *_rows(s, r, dev), _dense(w, _F32, dev), *_rows(dy, d, dev), *_rows(dsum, r, dev),
             *_rows(dx, d, dev), *_rows(dres, r, dev), _dense(dw, _F32, dev), *_area(ws, ws_bytes, dev),
             _raw_stream(dev) if stream is None else _stream(stream))


def gdn_conv_fwd(shape, x, w, bias, cu, s0, y, sT, stream=None) -> int:
    """y and, if given, the sequences' new states sT [B, W - 1, D]."""
    f, d, dev = _FN["gdn_conv_fwd"], _DTYPE.get(shape.io), _device()
    return f(_ref(shape), _flat(x, d, dev), _dense(w, _F32, dev), _dense(bias, _F32, dev), _dense(cu, _I32, dev),
             _dense(s0, d, dev), _flat(y, d, dev), _dense(sT, d, dev),
             _raw_stream(dev) if stream is None else _stream(stream))


def gdn_conv_workspace_bytes(shape) -> int:
    return load().gdn_conv_workspace_bytes(_ref(shape))


def gdn_conv_bwd(shape, x, w, bias, cu, s0, dy, dsT, dx, dw, dbias, ds0, ws, ws_bytes=None, stream=None) -> int:
    """The gradients of x, w [D, W], bias [D] and, if given, s0."""
    f, d, dev = _FN["gdn_conv_bwd"], _DTYPE.get(shape.io), _device()
    return f(_ref(shape), _flat(x, d, dev), _dense(w, _F32, dev), _dense(bias, _F32, dev), _dense(cu, _I32, dev),
             _dense(s0, d, dev), _flat(dy, d, dev), _dense(dsT, d, dev), _flat(dx, d, dev), _dense(dw, _F32, dev),
             _dense(dbias, _F32, dev), _dense(ds0, d, dev), *_area(ws, ws_bytes, dev),
             _raw_stream(dev) if stream is None else _stream(stream))


def gdn_conv_step(shape, x, w, bias, state, src, dst, y, stream=None) -> int:
    """y [B * T, D] of new tokens; state [slots, W - 1, D] is read at src [B] and written at dst [B] (None: src; None: b)."""
    f, d, dev = _FN["gdn_conv_step"], _DTYPE.get(shape.io), _device()
    return f(_ref(shape), _flat(x, d, dev), _dense(w, _F32, dev), _dense(bias, _F32, dev), _dense(state, d, dev),
             _dense(src, _I32, dev), _dense(dst, _I32, dev), _flat(y, d, dev),
             _raw_stream(dev) if stream is None else _stream(stream))


def gdn_scan_workspace_bytes(shape, backward) -> int:
    return load().gdn_scan_workspace_bytes(_ref(shape), int(backward))


def gdn_scan_saved_bytes(shape) -> int:
    """Bytes of what gdn_scan_fwd keeps for gdn_scan_bwd."""
    return load().gdn_scan_saved_bytes(_ref(shape))


def gdn_scan_fwd(shape, x, dt, z, Bm, Cm, A_log, D, dt_bias, cu, h0, y, hT, saved, ws, saved_bytes=None, ws_bytes=None,
                 stream=None) -> int:
    """y and, if given, the sequences' last states hT [B, D, N] and what gdn_scan_bwd needs (`saved`)."""
    f, d, dev = _FN["gdn_scan_fwd"], _DTYPE.get(shape.io), _device()
    return f(_ref(shape), _flat(x, d, dev), _flat(dt, d, dev), _flat(z, d, dev), _vectors(Bm, d, dev), _vectors(Cm, d, dev),
             _dense(A_log, _F32, dev), _dense(D, _F32, dev), _dense(dt_bias, _F32, dev), _dense(cu, _I32, dev),
             _dense(h0, _F32, dev), _flat(y, d, dev), _dense(hT, _F32, dev), *_area(saved, saved_bytes, dev),
             *_area(ws, ws_bytes, dev), _raw_stream(dev) if stream is None else _stream(stream))


def gdn_scan_bwd(shape, x, dt, z, Bm, Cm, A_log, D, dt_bias, cu, saved, dy, dhT, dx, ddt, dz, dBm, dCm, dA_log, dD, ddt_bias, dh0,
                 ws, saved_bytes=None, ws_bytes=None, stream=None) -> int:
    """The gradients of every input from dy, dhT and the forward's `saved`."""
    f, d, dev = _FN["gdn_scan_bwd"], _DTYPE.get(shape.io), _device()
    return f(_ref(shape), _flat(x, d, dev), _flat(dt, d, dev), _flat(z, d, dev), _vectors(Bm, d, dev), _vectors(Cm, d, dev),
             _dense(A_log, _F32, dev), _dense(D, _F32, dev), _dense(dt_bias, _F32, dev), _dense(cu, _I32, dev),
             *_area(saved, saved_bytes, dev), _flat(dy, d, dev), _dense(dhT, _F32, dev), _flat(dx, d, dev),
             _flat(ddt, d, dev), _flat(dz, d, dev), _vectors(dBm, d, dev), _vectors(dCm, d, dev), _dense(dA_log, _F32, dev),
             _dense(dD, _F32, dev), _dense(ddt_bias, _F32, dev), _dense(dh0, _F32, dev), *_area(ws, ws_bytes, dev),
             _raw_stream(dev) if stream is None else _stream(stream))


def gdn_scan_step(shape, x, dt, z, Bm, Cm, A_log, D, dt_bias, state, src, dst, y, stream=None) -> int:
    """y [B * T, D] of new tokens; state [slots, D, N] fp32 is read at src [B] and written at dst [B] (None: src; None: b)."""
    f, d, dev = _FN["gdn_scan_step"], _DTYPE.get(shape.io), _device()
    return f(_ref(shape), _flat(x, d, dev), _flat(dt, d, dev), _flat(z, d, dev), _vectors(Bm, d, dev), _vectors(Cm, d, dev),
             _dense(A_log, _F32, dev), _dense(D, _F32, dev), _dense(dt_bias, _F32, dev), _dense(state, _F32, dev),
             _dense(src, _I32, dev), _dense(dst, _I32, dev), _flat(y, d, dev),
             _raw_stream(dev) if stream is None else _stream(stream))
