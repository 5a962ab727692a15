"""Thin Python binding of the C ABI in ``include/qr_ops.h``: the operators of a
layer whose weights are held in the 4-bit block formats.

As in ``qr``: argument checks and marshalling only, the work runs in the HIP
kernels of ``libqr.so`` on the current (or the given) stream, and there is no
fallback path.  The operators have no gradient: an input that asks for one is
refused (ValueError) unless gradients are off (``torch.no_grad()``), so that none
is lost in silence.  Packing takes a weight that has one, as ``detach()`` does.
"""
import ctypes
import functools
import math

import torch

from . import qr as _qr
from .qr import DTYPES, _check, _fmt, _ptr, _stream, lib, qr_encode

WEIGHT_FORMATS = {4: 32, 20: 128, 36: 32}   # format id -> values that share a scale
ID_TYPES = {torch.int32: 4, torch.int64: 8}

_bound = None


def _lib():
    """``libqr.so`` with the signatures of the operators."""
    global _bound
    if _bound is None or _bound is not _qr._lib:
        L = lib()
        vp, sz, i = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
        L.qr_weight_bytes.restype = sz
        L.qr_weight_bytes.argtypes = [i, sz, sz]
        L.qr_linear.restype = i
        L.qr_linear.argtypes = [i, i, i, vp, sz, vp, vp, sz, sz, sz, sz, vp]
        L.qr_experts.restype = i
        L.qr_experts.argtypes = [i, i, i, vp, sz, sz, vp, vp, vp, vp, sz, sz, sz, sz, sz, vp]
        L.qr_route_workspace.restype = sz
        L.qr_route_workspace.argtypes = [sz, sz, sz]
        L.qr_route.restype = i
        L.qr_route.argtypes = [vp, i, vp, vp, vp, sz, sz, sz, vp, vp]
        L.qr_combine.restype = i
        L.qr_combine.argtypes = [i, vp, sz, sz, vp, vp, vp, sz, sz, sz, sz, vp]
        _bound = L
    return _bound


@functools.lru_cache(maxsize=1024)
def _weight_bytes(fid, rows, k):
    n = int(_lib().qr_weight_bytes(fid, rows, k))
    if not n:
        raise ValueError(f"no packed weight of format {fid}, {rows} rows of {k} values")
    return n


def qr_weight_bytes(fmt, rows, k):
    """Bytes of the packed form of a [rows, k] weight."""
    return _weight_bytes(_fmt(fmt), int(rows), int(k))


def qr_encode_weight(fmt, w, packed=None, stream=None):
    """Packs the fp16/bf16 device matrix ``w`` [rows, k] (or [experts, rows, k])
    as the products read it: rows padded with zeros to whole blocks, and the
    whole to a multiple of 2048 values, then ``qr_encode``."""
    fid = _fmt(fmt)
    if fid not in WEIGHT_FORMATS:
        raise ValueError(f"format {fmt!r} holds no weights (one of int4, asym4, fp4)")
    if w.dim() < 2:
        raise ValueError("w must have rows of k values")
    rows, k = math.prod(w.shape[:-1]), w.shape[-1]
    nbytes = _weight_bytes(fid, rows, k)
    group = WEIGHT_FORMATS[fid]
    kp = -(-k // group) * group
    n = -(-rows * kp // 2048) * 2048
    # every copy, that of a weight whose dimensions do not merge too, is made on the call's stream
    with torch.cuda.stream(stream) if stream is not None else torch.cuda.device(w.device):
        w = w.reshape(rows, k)
        if n != rows * k:
            flat = torch.zeros(n, dtype=w.dtype, device=w.device)
            flat[:rows * kp].view(rows, kp)[:, :k] = w
        else:
            flat = w.contiguous().view(-1)
    if packed is None:
        packed = _empty(w, (nbytes,), torch.uint8, stream)
    qr_encode(fid, flat, packed, stream)
    return packed


def _empty(like, shape, dtype, stream):
    """A new tensor on the device of ``like``, of the stream that will write it: the
    caching allocator hands memory on in the order of the stream that was current
    when it was taken."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def _matrix(t, name, rows, cols, device, dtype):
    """Address and row stride of a device matrix of ``cols`` neighbouring values a row."""
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dim() == 2):
        raise ValueError(f"{name} must be a device matrix")
    if t.get_device() != device:
        raise ValueError(f"{name} is on device {t.get_device()}, the call's tensors are on device {device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} is {t.dtype}, the call's dtype is {dtype}")
    if t.shape != (rows, cols):
        raise ValueError(f"{name} is {tuple(t.shape)}, the call needs {(rows, cols)}")
    return t.data_ptr(), _row_stride(t, name, rows, cols)


def _no_gradient(t, name):
    """Of an input with ``requires_grad`` (asked by the caller: a call is microseconds)."""
    if torch.is_grad_enabled():
        raise ValueError(f"{name} asks for a gradient, which this operator does not have: "
                         "detach it, or call under torch.no_grad()")


def _row_stride(t, name, rows, cols):
    ld, step = t.stride()
    if step != 1 and cols > 1:
        raise ValueError(f"the values of a row of {name} must be neighbours")
    if rows < 2:
        return cols
    if ld < cols:
        raise ValueError(f"the rows of {name} must not overlap")
    return ld


def _vector(t, name, numel, dtype, device):
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
    if t.numel() != numel:
        raise ValueError(f"{name} has {t.numel()} values, the call needs {numel}")
    return _ptr(t, name, 0, device)


@functools.lru_cache(maxsize=1024)
def _product_weight(fmt, experts, n, k, gated):
    """Format id and packed bytes of a product's weight."""
    fid = _fmt(fmt)
    if fid not in WEIGHT_FORMATS or n != int(n) or n < 1 or k < 1 or experts < 1:
        raise ValueError(f"no product of format {fmt!r} with n={n}, k={k}, {experts} expert(s)")
    return fid, _weight_bytes(fid, experts * n * (2 if gated else 1), k)


def _product(fn, fmt, x, w, n, gated, y, offsets, rows, stream):
    if not (isinstance(x, torch.Tensor) and x.is_cuda and x.dim() == 2):
        raise ValueError("x must be a device matrix")
    if x.requires_grad:
        _no_gradient(x, "x")
    dtype = x.dtype
    dt = DTYPES.get(dtype)
    if dt is None:
        raise ValueError(f"unsupported dtype {dtype}")
    tokens, k = x.shape
    dev = x.get_device()
    experts = 1 if offsets is None else offsets.numel() - 1
    fid, nbytes = _product_weight(fmt, experts, n, k, gated)
    ldx = _row_stride(x, "x", tokens, k)
    wp = _ptr(w, "w", nbytes, dev)
    slots = tokens if rows is None else rows.numel()
    if y is None:
        y = x.new_empty((slots, n)) if stream is None else _empty(x, (slots, n), dtype, stream)
        yp, ldy = y.data_ptr(), n
    else:
        yp, ldy = _matrix(y, "y", slots, n, dev, dtype)
    if offsets is None:
        st = _lib().qr_linear(fid, dt, gated, x.data_ptr(), ldx, wp, yp, ldy, slots, n, k, _stream(stream, dev))
    else:
        op = _vector(offsets, "offsets", experts + 1, torch.int32, dev)
        rp = None if rows is None else _vector(rows, "rows", slots, torch.int32, dev)
        st = _lib().qr_experts(fid, dt, gated, x.data_ptr(), ldx, tokens, wp, op, rp, yp, ldy, slots, experts, n, k,
                               _stream(stream, dev))
    if st:
        _check(fn, st)
    return y


def qr_linear(fmt, x, w, n, gated=False, y=None, stream=None):
    """``x`` [m, k] times the packed weight ``w`` [n, k] (``gated``: [2 n, k], the gate
    rows and then the up rows, for silu(gate) * up); returns ``y`` [m, n]."""
    return _product("qr_linear", fmt, x, w, n, gated, y, None, None, stream)


def qr_experts(fmt, x, w, n, offsets, rows=None, gated=False, y=None, stream=None):
    """The products of ``qr_linear`` with another weight for each group of rows.

    ``w`` is the packed [experts, n, k] weight (``gated``: [experts, 2 n, k]).  Row s of
    the result, for offsets[e] <= s < offsets[e + 1], is row ``rows[s]`` of ``x`` (row s
    without ``rows``) times the weight of expert e; the rows from offsets[-1] on are zero."""
    return _product("qr_experts", fmt, x, w, n, gated, y, offsets, rows, stream)


def qr_route(ids, experts, offsets=None, rows=None, pos=None, stream=None):
    """Plan of the router's choice ``ids`` [tokens, top] (int32 or int64; a number outside
    [0, experts) drops the slot): returns (offsets [experts + 1], rows [tokens * top],
    pos [tokens, top]), all int32.  Rows offsets[e] to offsets[e + 1] of the sorted order
    belong to expert e, sorted row s comes from token rows[s] (-1 past the last), and slot
    (t, j) went to row pos[t, j] (-1: dropped)."""
    if not (isinstance(ids, torch.Tensor) and ids.dim() == 2):
        raise ValueError("ids must be a device matrix [tokens, top]")
    idb = ID_TYPES.get(ids.dtype)
    if idb is None:
        raise ValueError(f"ids must be int32 or int64, not {ids.dtype}")
    tokens, top = ids.shape
    experts = int(experts)
    ip = _ptr(ids, "ids", 0)
    dev, slots = ids.get_device(), tokens * top
    if experts < 1 or top < 1:
        raise ValueError(f"no plan of {experts} expert(s), {top} a token")
    i32 = torch.int32
    if offsets is None:
        offsets = _empty(ids, (experts + 1,), i32, stream)
        op = offsets.data_ptr()
    else:
        op = _vector(offsets, "offsets", experts + 1, i32, dev)
    if rows is None:
        rows = _empty(ids, (slots,), i32, stream)
        rp = rows.data_ptr()
    else:
        rp = _vector(rows, "rows", slots, i32, dev)
    if pos is None:
        pos = _empty(ids, (tokens, top), i32, stream)
        pp = pos.data_ptr()
    else:
        pp = _vector(pos, "pos", slots, i32, dev)
    L = _lib()
    nbytes = _route_workspace(tokens, top, experts)
    ws = _empty(ids, (nbytes,), torch.uint8, stream) if nbytes else None  # scratch of this call
    st = L.qr_route(ip, idb, op, rp, pp, tokens, top, experts, ws.data_ptr() if nbytes else None, _stream(stream, dev))
    if st:
        _check("qr_route", st)
    return offsets, rows, pos


@functools.lru_cache(maxsize=1024)
def _route_workspace(tokens, top, experts):
    return int(_lib().qr_route_workspace(tokens, top, experts))


def qr_combine(y, pos, gates, out=None, stream=None):
    """out[t] = sum over j of gates[t, j] * y[pos[t, j]] (a position outside y: no term);
    ``pos`` int32 and ``gates`` fp32 are [tokens, top], ``y`` [slots, n]."""
    if not (isinstance(y, torch.Tensor) and y.is_cuda and y.dim() == 2):
        raise ValueError("y must be a device matrix")
    if not (isinstance(pos, torch.Tensor) and pos.dim() == 2):
        raise ValueError("pos must be a device matrix")
    if y.requires_grad:
        _no_gradient(y, "y")
    if gates.requires_grad:
        _no_gradient(gates, "gates")
    dtype = y.dtype
    dt = DTYPES.get(dtype)
    if dt is None:
        raise ValueError(f"unsupported dtype {dtype}")
    slots, n = y.shape
    tokens, top = pos.shape
    dev = y.get_device()
    yp, ldy = y.data_ptr(), _row_stride(y, "y", slots, n)
    if out is None:
        out = y.new_empty((tokens, n)) if stream is None else _empty(y, (tokens, n), dtype, stream)
        op, ldo = out.data_ptr(), n
    else:
        op, ldo = _matrix(out, "out", tokens, n, dev, dtype)
    pp = _vector(pos, "pos", tokens * top, torch.int32, dev)
    gp = _vector(gates, "gates", tokens * top, torch.float32, dev)
    st = _lib().qr_combine(dt, yp, ldy, slots, pp, gp, op, ldo, tokens, top, n, _stream(stream, dev))
    if st:
        _check("qr_combine", st)
    return out
