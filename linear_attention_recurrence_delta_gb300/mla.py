"""Latent attention (MLA): Python binding of the operators of ``include/gdn_mla.h``.

Like the recurrence's binding it only marshals arguments.  A tensor given as a view becomes its address and its row
and head strides, so slices of a projection's output (``q[..., :dn]``, ``kv[..., dn:]``) go in as they are: rows may
be one leading dimension ``[rows, heads, d]`` or ``[B, T, heads, d]`` whose first two collapse into rows.  A tensor
whose values are not laid out that way or not of the type that the call reads (torch.int32 for positions, offsets,
lengths and tables, torch.float32 for weights and statistics, the shape's io for the rest) raises ValueError; everything
else is checked by the library, which returns its status code.

One layer of a hybrid, between its projections (``gdn`` is this package)::

    p = gdn.make_mla_prep(N, H, dc, dr, "bf16", npos, page=64, B=B, npages=n, maxpages=m)
    gdn.check(gdn.gdn_mla_prep(p, kv, w, rot, pos, seq, table, q[..., dn:], cache, None, qr))    # into the cache
    s = gdn.make_mla_attn(B, H, Hkv, Tq, Tk, dn, dr, dv, "bf16", scale, Nq=Nq, Nk=Nk)
    ws = torch.empty(gdn.gdn_mla_workspace_bytes(s, 1), dtype=torch.uint8, device="cuda")
    gdn.check(gdn.gdn_mla_fwd(s, qn, qr, kn, kr, v, cu_q, cu_k, o, lse, ws))                      # prompts, training
    gdn.check(gdn.gdn_mla_bwd(s, qn, qr, kn, kr, v, cu_q, cu_k, o, lse, dO, dqn, dqr, dkn, dkr, dv, ws))
    c = gdn.make_mla_cache(B, T, H, dc, dr, 64, n, m, "bf16", scale)
    gdn.check(gdn.gdn_mla_decode(c, qc, qr, cache, table, lens, o, None, wd))                     # new tokens
"""
from __future__ import annotations

import ctypes

from . import _nbytes, _ptr, _stream, load


class gdn_mla_view_t(ctypes.Structure):
    _fields_ = [("p", ctypes.c_void_p), ("tok", ctypes.c_longlong), ("head", ctypes.c_longlong)]


class _Shape(ctypes.Structure):
    def __repr__(self):
        return f"{type(self).__name__}({', '.join(f'{k}={getattr(self, k)}' for k, _ in self._fields_)})"


def _ints(names):
    return [(n, ctypes.c_int) for n in names.split()]


class gdn_mla_prep_t(_Shape):
    _fields_ = _ints("N H dc dr io npos interleaved B page npages maxpages") + [("eps", ctypes.c_float)]


class gdn_mla_attn_t(_Shape):
    _fields_ = _ints("B H Hkv Tq Tk dn dr dv causal io Nq Nk") + [("scale", ctypes.c_float)]


class gdn_mla_cache_t(_Shape):
    _fields_ = _ints("B T H dc dr page npages maxpages io") + [("scale", ctypes.c_float)]


_IO = {"f32": 0, "bf16": 1}


def make_mla_prep(N, H, dc, dr, io="bf16", npos=0, eps=1e-6, interleaved=False, B=0, page=0, npages=0, maxpages=0):
    """npos: positions lie below it; a shape with tokens and without it is refused by the calls."""
    return gdn_mla_prep_t(int(N), int(H), int(dc), int(dr), _IO.get(io, io), int(npos), int(bool(interleaved)), int(B),
                          int(page), int(npages), int(maxpages), float(eps))


def make_mla_attn(B, H, Hkv, Tq, Tk, dn, dr, dv, io="bf16", scale=None, causal=True, Nq=None, Nk=None):
    """scale: 1 / sqrt(dn + dr) if not given; Nq, Nk: rows of packed tensors (B * Tq, B * Tk if not given)."""
    scale = (dn + dr) ** -0.5 if scale is None else scale
    return gdn_mla_attn_t(int(B), int(H), int(Hkv), int(Tq), int(Tk), int(dn), int(dr), int(dv), int(bool(causal)),
                          _IO.get(io, io), int(B * Tq if Nq is None else Nq), int(B * Tk if Nk is None else Nk), float(scale))


def make_mla_cache(B, T, H, dc, dr, page, npages, maxpages, io="bf16", scale=1.0):
    return gdn_mla_cache_t(int(B), int(T), int(H), int(dc), int(dr), int(page), int(npages), int(maxpages),
                           _IO.get(io, io), float(scale))


_F32 = _I32 = _DTYPE = None      # torch's types; by gdn_dtype_t


def declare(lib):
    """Signatures of the library's functions (called once, when it is loaded)."""
    global _F32, _I32, _DTYPE
    import torch
    _F32, _I32, _DTYPE = torch.float32, torch.int32, {0: torch.float32, 1: torch.bfloat16}
    vp, ll, sz, vw = ctypes.c_void_p, ctypes.c_longlong, ctypes.c_size_t, ctypes.POINTER(gdn_mla_view_t)
    sp, sa, sc = (ctypes.POINTER(t) for t in (gdn_mla_prep_t, gdn_mla_attn_t, gdn_mla_cache_t))
    for name, args, res in (
            ("gdn_mla_prep", [sp, vp, ll, vp, vp, vp, vp, vp, vw, vw, vw, vw, vp], ctypes.c_int),
            ("gdn_mla_prep_workspace_bytes", [sp], sz),
            ("gdn_mla_prep_bwd", [sp, vp, ll, vp, vp, vp, vw, vw, vw, vp, ll, vp, vw, vp, sz, vp], ctypes.c_int),
            ("gdn_mla_workspace_bytes", [sa, ctypes.c_int], sz),
            ("gdn_mla_fwd", [sa, vw, vw, vw, vw, vw, vp, vp, vp, vp, vp, sz, vp], ctypes.c_int),
            ("gdn_mla_bwd", [sa, vw, vw, vw, vw, vw, vp, vp, vp, vp, vp, vw, vw, vw, vw, vw, vp, sz, vp], ctypes.c_int),
            ("gdn_mla_decode_workspace_bytes", [sc], sz),
            ("gdn_mla_decode", [sc, vw, vw, vp, vp, vp, vp, vp, vp, sz, vp], ctypes.c_int)):
        f = getattr(lib, name)
        f.argtypes, f.restype = args, res


_ref = ctypes.byref


def _view(t, heads=True):
    """A tensor as (address, row stride, head stride); None and a ready view pass through."""
    if t is None or isinstance(t, gdn_mla_view_t):
        return t
    shape, stride = t.shape, t.stride()
    lead = len(shape) - (2 if heads else 1)          # dimensions that count rows
    if lead not in (1, 2):
        raise ValueError(f"a view is [rows, {'heads, ' if heads else ''}d] or [B, T, ...]: got {tuple(shape)}")
    if shape[-1] > 1 and stride[-1] != 1:
        raise ValueError("the last dimension of a view has to be contiguous")
    if lead == 2 and shape[0] > 1 and shape[1] > 0 and stride[0] != shape[1] * stride[1]:
        raise ValueError("the first two dimensions of a view have to collapse into rows")
    tok = stride[lead - 1]
    if lead == 2 and shape[1] == 1:
        tok = stride[0]
    if all(n == 1 for n in shape[:lead]):            # one row: its stride means nothing
        tok = -(-(shape[lead] * stride[lead] if heads else shape[-1]) // 8) * 8
    return gdn_mla_view_t(t.data_ptr(), tok, stride[lead] if heads else tok)


def _typed(t, dtype):
    """For a tensor that is not of the wanted type (None: any will do)."""
    if dtype is not None:
        raise ValueError(f"a tensor of {dtype} is wanted here, not of {t.dtype}")


# A decoding step waits for these calls' host time, so the common layouts take a short way (half a microsecond a view).

def _heads(t, dtype=None):
    """[rows, heads, d] or [B, T, heads, d] by reference."""
    if t is None:
        return None
    if type(t) is not gdn_mla_view_t:
        if t.dtype is not dtype:
            _typed(t, dtype)
        s = t.stride()
        if len(s) == 3 and s[2] == 1 and s[0] % 8 == 0 and s[0] > 0:
            return _ref(gdn_mla_view_t(t.data_ptr(), s[0], s[1]))
        if len(s) == 4 and t.is_contiguous():
            n = t.shape
            return _ref(gdn_mla_view_t(t.data_ptr(), n[2] * n[3], n[3]))
        t = _view(t)
    return _ref(t)


def _flat(t, dtype=None):
    """[rows, d] by reference."""
    if t is None:
        return None
    if type(t) is not gdn_mla_view_t:
        if t.dtype is not dtype:
            _typed(t, dtype)
    return _ref(_view(t, heads=False))


def _size(ws, ws_bytes):
    return _nbytes(ws) if ws_bytes is None and ws is not None else (ws_bytes or 0)


def _rows(t, dtype=None):
    """A tensor of contiguous rows as (address, row stride)."""
    if t is None or isinstance(t, int):
        return t, 0
    if t.dtype is not dtype:
        _typed(t, dtype)
    s = t.stride()
    if len(s) == 2 and s[1] == 1 and s[0] % 8 == 0 and s[0] > 0:
        return t.data_ptr(), s[0]
    v = _view(t, heads=False)
    return v.p, v.tok


def _dense(t, dtype=None):
    """The address of a contiguous tensor."""
    if t is None or type(t) is int:
        return t
    if t.dtype is not dtype:
        _typed(t, dtype)
    if not t.is_contiguous():
        raise ValueError("o, dO, lse, cache, table, lengths, offsets, positions and workspaces are contiguous")
    return t.data_ptr()


def gdn_mla_prep(shape, kv, w, rot, pos, seq, table, qr, lat, kr, qr_out, stream=None) -> int:
    """Norm, rotate and write: into the paged cache `lat` (shape.page > 0; kr None), or to dense rows lat, kr."""
    f, d = load().gdn_mla_prep, _DTYPE.get(shape.io)
    rows = _ref(gdn_mla_view_t(_dense(lat, d), 0, 0)) if shape.page > 0 else _flat(lat, d)
    return f(_ref(shape), *_rows(kv, d), _dense(w, _F32), _dense(rot, _F32), _dense(pos, _I32), _dense(seq, _I32),
             _dense(table, _I32), _heads(qr, d), rows, _flat(kr, d), _heads(qr_out, d), _stream(stream))


def gdn_mla_prep_workspace_bytes(shape) -> int:
    return load().gdn_mla_prep_workspace_bytes(_ref(shape))


def gdn_mla_prep_bwd(shape, kv, w, rot, pos, dlat, dkr, dqr, dkv, dw, dqr_out, ws, ws_bytes=None, stream=None) -> int:
    """Gradients of the dense form: dkv [N, dc + dr], dw [dc] fp32 and dqr_out."""
    f, d = load().gdn_mla_prep_bwd, _DTYPE.get(shape.io)
    return f(_ref(shape), *_rows(kv, d), _dense(w, _F32), _dense(rot, _F32), _dense(pos, _I32), _flat(dlat, d), _flat(dkr, d),
             _heads(dqr, d), *_rows(dkv, d), _dense(dw, _F32), _heads(dqr_out, d), _ptr(ws), _size(ws, ws_bytes),
             _stream(stream))


def gdn_mla_workspace_bytes(shape, backward) -> int:
    return load().gdn_mla_workspace_bytes(_ref(shape), int(backward))


def gdn_mla_fwd(shape, qn, qr, kn, kr, v, cu_q, cu_k, o, lse, ws, ws_bytes=None, stream=None) -> int:
    """o and, if given, lse [H, Nq] fp32."""
    f, d = load().gdn_mla_fwd, _DTYPE.get(shape.io)
    return f(_ref(shape), _heads(qn, d), _heads(qr, d), _heads(kn, d), _flat(kr, d), _heads(v, d), _dense(cu_q, _I32),
             _dense(cu_k, _I32), _dense(o, d), _dense(lse, _F32), _ptr(ws), _size(ws, ws_bytes), _stream(stream))


def gdn_mla_bwd(shape, qn, qr, kn, kr, v, cu_q, cu_k, o, lse, dO, dqn, dqr, dkn, dkr, dv, ws, ws_bytes=None,
                stream=None) -> int:
    """The gradients of qn, qr, kn, kr and v from dO and the forward's o and lse."""
    f, d = load().gdn_mla_bwd, _DTYPE.get(shape.io)
    return f(_ref(shape), _heads(qn, d), _heads(qr, d), _heads(kn, d), _flat(kr, d), _heads(v, d), _dense(cu_q, _I32),
             _dense(cu_k, _I32), _dense(o, d), _dense(lse, _F32), _dense(dO, d), _heads(dqn, d), _heads(dqr, d),
             _heads(dkn, d), _flat(dkr, d), _heads(dv, d), _ptr(ws), _size(ws, ws_bytes), _stream(stream))


def gdn_mla_decode_workspace_bytes(shape) -> int:
    return load().gdn_mla_decode_workspace_bytes(_ref(shape))


def gdn_mla_decode(shape, qc, qr, cache, table, lens, o, lse, ws, ws_bytes=None, stream=None) -> int:
    """o [B, T, H, dc] and, if given, lse [B, T, H] fp32 of new tokens over the paged latent cache."""
    f, d = load().gdn_mla_decode, _DTYPE.get(shape.io)
    return f(_ref(shape), _heads(qc, d), _heads(qr, d), _dense(cache, d), _dense(table, _I32), _dense(lens, _I32), _dense(o, d),
             _dense(lse, _F32), _ptr(ws), _size(ws, ws_bytes), _stream(stream))
