"""Thin Python binding of the C ABI in ``include/qr_rows.h``: the operators of a layer
whose activations and weights are held in rows of 8 bits, the norm in front of it and
the router's choice.

As in ``qr_ops``: argument checks and marshalling only, the work runs in the HIP kernels
of ``libqr.so`` on the current (or the given) stream, there is no fallback path, and an
input that asks for a gradient is refused unless gradients are off.  (``qr_encode_rows``
takes one that has one, as ``detach()`` does: it packs weights too.)
"""
import ctypes
import functools
import math

import torch

from . import qr as _qr
from .qr import DTYPES, _check, _ptr, _stream, lib
from .qr_ops import _empty, _matrix, _no_gradient, _row_stride, _vector

MAX_ROW_K = 130944
ROW_RUN = 128          # codes that a row is padded to a multiple of
LOGIT_DTYPES = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}
SCORES = {"softmax": 0, "sigmoid": 1}

_bound = None


def _lib():
    """``libqr.so`` with the signatures of the operators."""
    global _bound
    if _bound is None or _bound is not _qr._lib:
        L = lib()
        vp, sz, i, f = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_float
        L.qr_row_bytes.restype = sz
        L.qr_row_bytes.argtypes = [sz, sz]
        L.qr_encode_rows.restype = i
        L.qr_encode_rows.argtypes = [i, vp, sz, vp, vp, sz, sz, vp]
        L.qr_decode_rows.restype = i
        L.qr_decode_rows.argtypes = [i, vp, vp, vp, sz, sz, sz, vp]
        L.qr_norm.restype = i
        L.qr_norm.argtypes = [i, vp, sz, vp, sz, vp, f, vp, sz, vp, sz, vp, vp, sz, sz, vp]
        L.qr_linear8.restype = i
        L.qr_linear8.argtypes = [i, i, vp, vp, vp, vp, vp, sz, sz, sz, sz, vp]
        L.qr_experts8.restype = i
        L.qr_experts8.argtypes = [i, i, vp, vp, sz, vp, vp, vp, vp, vp, sz, sz, sz, sz, sz, vp]
        L.qr_choose.restype = i
        L.qr_choose.argtypes = [i, i, vp, sz, vp, sz, sz, i, i, f, vp, vp, sz, sz, sz, vp]
        _bound = L
    return _bound


@functools.lru_cache(maxsize=1024)
def _row_bytes(rows, k):
    n = int(_lib().qr_row_bytes(rows, k))
    if not n:
        raise ValueError(f"no 8-bit rows of {rows} x {k} values (k is at most {MAX_ROW_K})")
    return n


def qr_row_bytes(rows, k):
    """Bytes of the codes of ``rows`` 8-bit rows of ``k`` values."""
    return _row_bytes(int(rows), int(k))


# The current device's number without the checks of torch.cuda.current_device() (a call is microseconds).
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _call(device, fn, *args):
    """The library's call with the tensors' device current: a launch goes to the current one."""
    f = getattr(_lib(), fn)
    if _current_device() == device:
        st = f(*args)
    else:
        with torch.cuda.device(device):
            st = f(*args)
    if st:
        _check(fn, st)


def _dtype(dtype):
    dt = DTYPES.get(dtype)
    if dt is None:
        raise ValueError(f"unsupported dtype {dtype}")
    return dt


def _width(k):
    if not 1 <= k <= MAX_ROW_K:
        raise ValueError(f"rows of {k} values: 1 to {MAX_ROW_K} are possible")
    return -(-k // ROW_RUN) * ROW_RUN


def _device(t, name):
    dev = t.get_device() if isinstance(t, torch.Tensor) else -1
    if dev < 0:
        raise ValueError(f"{name} must be a device tensor")
    return dev


def _values(t, name, numel, dtype, device):
    """Address of a contiguous device tensor of ``numel`` values."""
    if t.dtype is dtype and t.get_device() == device and t.numel() == numel and t.is_contiguous():
        return t.data_ptr()
    return _vector(t, name, numel, dtype, device)     # says what is wrong


def _rows(t, name, rows, k, dtype, device):
    """Address and row stride of a device matrix."""
    if t.dtype is dtype and t.get_device() == device and t.shape == (rows, k):
        ld, step = t.stride()
        if step == 1 and rows > 1 and ld >= k:
            return t.data_ptr(), ld
        if rows == 1 and (step == 1 or k == 1):
            return t.data_ptr(), k
    return _matrix(t, name, rows, k, device, dtype)   # says what is wrong, if anything is


def _codes(t, s, name, device=None):
    """Addresses of 8-bit rows, their device and shape: contiguous int8 codes [..., whole runs] and fp32 scales."""
    dev = _device(t, f"the codes of {name}") if device is None else device
    shape = t.shape
    if t.dtype is not torch.int8 or len(shape) < 2:
        raise ValueError(f"the codes of {name} must be int8 rows")
    k = shape[-1]
    if k % ROW_RUN or not k:
        raise ValueError(f"the codes of {name} have rows of {k}: whole runs of {ROW_RUN}, padded with zeros")
    if not t.is_contiguous() or t.get_device() != dev:
        _ptr(t, f"the codes of {name}", 0, device)
    if s.requires_grad:
        _no_gradient(s, f"a scale of {name}")
    return t.data_ptr(), _values(s, f"the scales of {name}", t.numel() // k, torch.float32, dev), dev, shape


def _new_codes(like, shape, k, codes, scales, stream, device):
    """Given or new codes and scales of rows of k values."""
    width, rows = _width(k), math.prod(shape)
    if codes is None:
        codes = _empty(like, (*shape, width), torch.int8, stream)
        cp = codes.data_ptr()
    elif codes.dtype != torch.int8 or codes.shape != (*shape, width):
        raise ValueError(f"codes is {codes.dtype} {tuple(codes.shape)}, the call needs int8 {(*shape, width)}")
    else:
        cp = _ptr(codes, "codes", 0, device)
    if scales is None:
        scales = _empty(like, shape, torch.float32, stream)
        sp = scales.data_ptr()
    else:
        sp = _vector(scales, "scales", rows, torch.float32, device)
    return codes, scales, cp, sp


def qr_encode_rows(x, codes=None, scales=None, stream=None):
    """8-bit rows of the fp16/bf16 device tensor ``x`` [..., k]: returns (codes int8 [..., k rounded
    up to whole runs of 128], scales fp32 [...]).  A weight [n, k] or [experts, n, k] has a scale for each
    row of n, a matrix of tokens one for each token."""
    dev = _device(x, "x")
    if x.dim() < 2:
        raise ValueError("x must have rows of values")
    dt, k, shape = _dtype(x.dtype), x.shape[-1], x.shape[:-1]
    _width(k)
    rows = math.prod(shape)
    if x.dim() > 2:
        # a copy, if the dimensions do not merge, is made on the call's stream
        with torch.cuda.stream(stream) if stream is not None else torch.cuda.device(dev):
            x = x.detach().reshape(rows, k)
    ldx = _row_stride(x, "x", rows, k)
    codes, scales, cp, sp = _new_codes(x, shape, k, codes, scales, stream, dev)
    _call(dev, "qr_encode_rows", dt, x.data_ptr(), ldx, cp, sp, rows, k, _stream(stream, dev))
    return codes, scales


def qr_decode_rows(codes, scales, k, dtype, y=None, stream=None):
    """The values [..., k] of ``dtype`` that 8-bit rows stand for."""
    dt, k = _dtype(dtype), int(k)
    cp, sp, dev, shape = _codes(codes, scales, "the rows")
    if _width(k) != shape[-1]:
        raise ValueError(f"rows of {codes.shape[-1]} codes do not hold {k} values")
    rows = scales.numel()
    if y is None:
        y = _empty(codes, (*shape[:-1], k), dtype, stream)
        yp, ldy = y.data_ptr(), k
    elif len(shape) == 2:
        yp, ldy = _rows(y, "y", rows, k, dtype, dev)
    else:
        if y.dtype != dtype or y.shape != (*shape[:-1], k):
            raise ValueError(f"y is {y.dtype} {tuple(y.shape)}, the call needs {dtype} {(*shape[:-1], k)}")
        yp, ldy = _ptr(y, "y", 0, dev), k
    _call(dev, "qr_decode_rows", dt, cp, sp, yp, ldy, rows, k, _stream(stream, dev))
    return y


def _norm(x, weight, eps, residual, total, y, codes, scales, with_output, with_rows, stream):
    dev = _device(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be a device matrix")
    if x.requires_grad:
        _no_gradient(x, "x")
    if weight.requires_grad:
        _no_gradient(weight, "weight")
    dtype = x.dtype
    dt = _dtype(dtype)
    rows, k = x.shape
    _width(k)
    if not eps >= 0:
        raise ValueError(f"eps is {eps}, must not be negative")
    ldx = _row_stride(x, "x", rows, k)
    wp = _values(weight, "weight", k, dtype, dev)
    rp = tp = yp = cp = sp = None
    ldr = ldt = ldy = k
    if residual is not None:
        if residual.requires_grad:
            _no_gradient(residual, "residual")
        rp, ldr = _rows(residual, "residual", rows, k, dtype, dev)
        if total is None:
            total = x.new_empty((rows, k)) if stream is None else _empty(x, (rows, k), dtype, stream)
            tp = total.data_ptr()
        else:
            tp, ldt = _rows(total, "total", rows, k, dtype, dev)
    elif total is not None:
        raise ValueError("total is x itself without a residual")
    if y is not None:
        yp, ldy = _rows(y, "y", rows, k, dtype, dev)
    elif with_output:
        y = x.new_empty((rows, k)) if stream is None else _empty(x, (rows, k), dtype, stream)
        yp = y.data_ptr()
    if with_rows:
        codes, scales, cp, sp = _new_codes(x, (rows,), k, codes, scales, stream, dev)
    _call(dev, "qr_norm", dt, x.data_ptr(), ldx, rp, ldr, wp, eps, tp, ldt, yp, ldy, cp, sp, rows, k, _stream(stream, dev))
    return y, total, codes, scales


def qr_norm(x, weight, eps=1e-6, residual=None, y=None, total=None, stream=None):
    """Root-mean-square norm of the rows of h = ``x`` + ``residual``: returns (y, total), where
    y = h / sqrt(mean(h^2) + eps) * ``weight`` and total is h, the next norm's residual (None without
    one).  ``total`` may be ``x`` or ``residual`` itself, ``y`` that of them which ``total`` is not."""
    y, total, _, _ = _norm(x, weight, eps, residual, total, y, None, None, True, False, stream)
    return y, total


def qr_norm_rows(x, weight, eps=1e-6, residual=None, with_output=False, codes=None, scales=None, y=None, total=None,
                 stream=None):
    """The norm of ``qr_norm`` as 8-bit rows, made of y before it is rounded: returns (codes, scales,
    total, y); y is None unless it is given or asked for by ``with_output``."""
    y, total, codes, scales = _norm(x, weight, eps, residual, total, y, codes, scales, with_output, True, stream)
    return codes, scales, total, y


def _product8(fn, x, xs, w, ws, dtype, gated, y, offsets, rows, stream):
    dt = DTYPES.get(dtype)
    if dt is None:
        raise ValueError(f"unsupported dtype {dtype}")
    xp, xsp, dev, xshape = _codes(x, xs, "x")
    wp, wsp, _, wshape = _codes(w, ws, "w", dev)
    if len(xshape) != 2 or len(wshape) != (2 if offsets is None else 3):
        raise ValueError(f"x has 2 dimensions and w {2 if offsets is None else 3}, not {len(xshape)} and {len(wshape)}")
    tokens, k = xshape
    n = wshape[-2]
    if wshape[-1] != k:
        raise ValueError(f"rows of {k} codes times rows of {wshape[-1]}")
    if gated:
        if n % 2:
            raise ValueError(f"a gated weight has as many gate as up rows, not {n} in all")
        n //= 2
    slots = tokens if rows is None else rows.numel()
    if y is None:
        y = x.new_empty((slots, n), dtype=dtype) if stream is None else _empty(x, (slots, n), dtype, stream)
        yp, ldy = y.data_ptr(), n
    else:
        yp, ldy = _rows(y, "y", slots, n, dtype, dev)
    if offsets is None:
        _call(dev, fn, dt, gated, xp, xsp, wp, wsp, yp, ldy, slots, n, k, _stream(stream, dev))
    else:
        experts = wshape[0]
        op = _values(offsets, "offsets", experts + 1, torch.int32, dev)
        rp = None if rows is None else _values(rows, "rows", slots, torch.int32, dev)
        _call(dev, fn, dt, gated, xp, xsp, tokens, wp, wsp, op, rp, yp, ldy, slots, experts, n, k,
                   _stream(stream, dev))
    return y


def qr_linear8(x, xs, w, ws, dtype, gated=False, y=None, stream=None):
    """The 8-bit rows ``x`` (codes [m, k], scales ``xs`` [m]) times the weight ``w`` (codes [n, k], scales ``ws``
    [n]; ``gated``: 2 n rows, the gate rows and then the up rows, for silu(gate) * up); returns ``y`` [m, n] of
    ``dtype``."""
    return _product8("qr_linear8", x, xs, w, ws, dtype, gated, y, None, None, stream)


def qr_experts8(x, xs, w, ws, offsets, dtype, rows=None, gated=False, y=None, stream=None):
    """The products of ``qr_linear8`` with another weight for each group of rows.

    ``w`` is [experts, n, k] codes (``gated``: [experts, 2 n, k]), ``ws`` their scales.  Row s of the result, for
    offsets[e] <= s < offsets[e + 1], is row ``rows[s]`` of ``x`` (row s without ``rows``) times the weight of expert e;
    the rows from offsets[-1] on are zero."""
    return _product8("qr_experts8", x, xs, w, ws, dtype, gated, y, offsets, rows, stream)


def qr_choose(logits, top, score="softmax", bias=None, groups=1, top_groups=1, group_best=1, renormalise=True,
              factor=1.0, gates=None, ids=None, stream=None):
    """A router's choice: the ``top`` experts of each token by score (softmax or sigmoid of ``logits`` [tokens, experts],
    fp16, bf16 or fp32) plus ``bias`` (fp32, for the choice only), largest first, ties to the lower number.  With
    ``groups``, of the ``top_groups`` groups of neighbouring experts whose ``group_best`` largest ranks sum to most.
    Returns (gates fp32 [tokens, top], ids int32 [tokens, top]): the scores of the chosen, divided by their sum if
    ``renormalise``, times ``factor``.  A logit of -inf or NaN takes its expert out; where fewer than ``top`` are left
    the last ids are -1, with gates of 0, as ``qr_route`` and ``qr_combine`` drop them."""
    dev = _device(logits, "logits")
    if logits.dim() != 2:
        raise ValueError("logits must be a device matrix [tokens, experts]")
    dt = LOGIT_DTYPES.get(logits.dtype)
    if dt is None or score not in SCORES:
        raise ValueError(f"no choice by {score!r} of logits of {logits.dtype}")
    if logits.requires_grad:
        _no_gradient(logits, "logits")
    if bias is not None and bias.requires_grad:
        _no_gradient(bias, "bias")
    tokens, experts = logits.shape
    top = int(top)
    if top < 1 or experts < 1:
        raise ValueError(f"no choice of {top} of {experts} experts")
    ldl = _row_stride(logits, "logits", tokens, experts)
    bp = None if bias is None else _values(bias, "bias", experts, torch.float32, dev)
    if gates is None:
        gates = _empty(logits, (tokens, top), torch.float32, stream)
        gp = gates.data_ptr()
    else:
        gp = _vector(gates, "gates", tokens * top, torch.float32, dev)
    if ids is None:
        ids = _empty(logits, (tokens, top), torch.int32, stream)
        ip = ids.data_ptr()
    else:
        ip = _vector(ids, "ids", tokens * top, torch.int32, dev)
    _call(dev, "qr_choose", dt, SCORES[score], logits.data_ptr(), ldl, bp, int(groups), int(top_groups),
               int(group_best), bool(renormalise), float(factor), gp, ip, tokens, experts, top, _stream(stream, dev))
    return gates, ids
