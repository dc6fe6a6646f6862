"""Python binding of the token-table and norm calls of libzero_mi355x.so,
declared in include/zero_layers.h: the same names, argument marshalling only.

Sizes, types and strides are the tensors': arrays of rows are tensors of two
dimensions whose last one is consecutive (a slice of columns passes its
stride); tokens are int32 or int64, of any shape, without gaps. Outputs and
workspaces are the caller's, on the inputs' device, which has to be the current
one. Streams and errors are those of ``zero``.
"""

from __future__ import annotations

import ctypes
import struct

from . import zero
from .tensors import ZERO_BF16, ZERO_F32  # noqa: F401 (the types of a call's arrays)

ZERO_I32 = 2
ZERO_I64 = 3
ZERO_LAYER_ROWS = 16777215
ZERO_LAYER_DIM = 1048576
ZERO_LAYER_ELEMS = 34359738368

_VP = ctypes.c_void_p
_I64 = ctypes.c_int64
_I32 = ctypes.c_int32


class zero_norm_args(ctypes.Structure):
    _fields_ = [(k, _VP) for k in ("x", "residual", "total", "y", "weight", "bias", "mean", "rstd")] + \
               [(k, _I64) for k in ("n", "dim", "x_stride", "residual_stride", "total_stride", "y_stride")] + \
               [("eps", ctypes.c_double)] + [(k, _I32) for k in ("type", "weight_type", "rms", "reserved")]


class zero_norm_grad_args(ctypes.Structure):
    _fields_ = [(k, _VP) for k in ("d_y", "x", "d_total", "d_x", "weight", "mean", "rstd", "d_weight", "d_bias")] + \
               [(k, _I64) for k in ("n", "dim", "d_y_stride", "x_stride", "d_total_stride", "d_x_stride")] + \
               [(k, _I32) for k in ("type", "weight_type", "grad_type", "rms", "accumulate", "reserved")]


_SIGNATURES = {
    "zero_embedding": (ctypes.c_int, [_VP, _I32, _I64, _VP, _I32, _I64, _I64, ctypes.c_double, _VP, _I32, _I64, _VP]),
    "zero_token_order_bytes": (ctypes.c_size_t, [_I64, _I64]),
    "zero_token_order": (ctypes.c_int, [_VP, _I32, _I64, _I64, _VP, ctypes.c_size_t, _VP]),
    "zero_embedding_grad_workspace_bytes": (ctypes.c_size_t, [_I64, _I64]),
    "zero_embedding_grad": (ctypes.c_int, [_VP, _I64, _I64, _I64, _VP, _I32, _I64, ctypes.c_double, _VP, _I32, _I64,
                                           _I64, _I32, _VP, ctypes.c_size_t, _VP]),
    "zero_norm": (ctypes.c_int, [_VP, _VP]),
    "zero_norm_grad_workspace_bytes": (ctypes.c_size_t, [_I64, _I64]),
    "zero_norm_grad": (ctypes.c_int, [_VP, _VP, ctypes.c_size_t, _VP]),
}

_lib = None


def library():
    """The library's handle with these calls' signatures set."""
    global _lib
    if _lib is None:
        lib = zero.library()
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


_torch = _C = _TYPES = _IDS = _F32 = None


def _load():
    """torch and the library, at the first call."""
    global _torch, _C, _TYPES, _IDS, _F32
    import torch
    library()
    _TYPES = {torch.bfloat16: ZERO_BF16, torch.float32: ZERO_F32}
    _IDS = {torch.int32: ZERO_I32, torch.int64: ZERO_I64}
    _F32 = (torch.float32,)
    _C, _torch = torch._C, torch


# ctypes cuts an integer to the 64 bits of its argument: one beyond them is refused here.
_TOP = 1 << 63


def _fits(k, what):
    if not -_TOP <= k < _TOP:
        raise ValueError(f"{what} = {k} is beyond the limits of include/zero_layers.h")


def _sized(name, *sizes):
    """Bytes of an order or a workspace."""
    fit = all(-_TOP <= k < _TOP for k in sizes)
    nbytes = int(getattr(_lib or library(), name)(*sizes)) if fit else 0
    if nbytes == 0:
        raise ValueError(f"{name}: sizes {sizes} outside the limits of include/zero_layers.h")
    return nbytes


# The checks cost a call 0.5 us a tensor, of the 4 to 7 that it takes in all: each tensor's
# attributes are read once, and what is wrong is found out only where something is.

def _device():
    """The current device, where the library's launches go."""
    if _torch is None:
        _load()
    try:
        return _C._cuda_getDevice()
    except RuntimeError:        # no device: every tensor is refused
        return -1


def _refuse(t, what, dev, dtypes):
    """The error of a tensor that is not on the current device or not of these types."""
    if not getattr(t, "is_cuda", False):
        raise TypeError(f"{what}: device memory expected, got {type(t).__name__}"
                        f"{' on ' + str(t.device) if hasattr(t, 'device') else ''}")
    if t.get_device() != dev:
        raise ValueError(f"{what} is on {t.device}, the current device is {dev}")
    if dtypes is not None and t.dtype not in dtypes:
        raise TypeError(f"{what}: {' or '.join(str(d) for d in dtypes)} expected, got {t.dtype}")


def _rows(t, what, dev, shape, dtypes):
    """(address, stride) of an array of rows of this shape (a pair; None: any)."""
    try:
        step, one = t.stride()
        size = t.shape
        if t.get_device() == dev >= 0 and t.dtype in dtypes and (shape is None or size == shape):
            if one == 1 or size[1] <= 1:
                return t.data_ptr(), step if size[0] > 1 else size[1]
    except (AttributeError, ValueError, TypeError):      # no tensor, or not of two dimensions
        pass
    _refuse(t, what, dev, dtypes)
    if t.dim() != 2 or (shape is not None and t.shape != shape):
        raise ValueError(f"{what}: {'two dimensions' if shape is None else tuple(shape)} expected, got {tuple(t.shape)}")
    raise ValueError(f"{what}: the elements of a row have to be consecutive")


def _flat(t, what, dev, count, dtypes):
    """Address of an array without gaps of `count` elements."""
    try:
        if t.get_device() == dev >= 0 and t.dtype in dtypes and t.numel() == count and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(t, what, dev, dtypes)
    if t.numel() != count:
        raise ValueError(f"{what}: {t.numel()} elements, {count} expected")
    raise ValueError(f"{what}: a contiguous tensor is expected")


def _memory(t, what, dev):
    """(address, bytes) of an order or a workspace, of any type."""
    try:
        if t.get_device() == dev >= 0 and t.is_contiguous():
            return t.data_ptr(), t.nbytes
    except AttributeError:
        pass
    _refuse(t, what, dev, None)
    raise ValueError(f"{what}: a contiguous tensor is expected")


def _stream(stream, dev):
    return _C._cuda_getCurrentRawStream(dev) if stream is None else zero._stream(stream)


def _tokens(tokens, dev):
    """(address, number) of the tokens."""
    n = tokens.numel() if hasattr(tokens, "numel") else 0
    return _flat(tokens, "tokens", dev, n, _IDS), n


def zero_embedding(tokens, table, out, scale: float = 1.0, stream=None):
    """``out`` [number of tokens, dim] = scale * rows of ``table`` [rows, dim]."""
    dev = _device()
    ids, n = _tokens(tokens, dev)
    src, step = _rows(table, "table", dev, None, _TYPES)
    rows, dim = table.shape
    if step != dim:
        raise ValueError("table: rows without gaps are expected")
    dst, stride = _rows(out, "out", dev, (n, dim), _TYPES)
    rc = _lib.zero_embedding(ids, _IDS[tokens.dtype], n, src, _TYPES[table.dtype], rows, dim, scale, dst,
                             _TYPES[out.dtype], stride, _stream(stream, dev))
    if rc:
        zero._check("zero_embedding", rc)


def zero_token_order_bytes(n: int, rows: int) -> int:
    return _sized("zero_token_order_bytes", n, rows)


def zero_token_order(tokens, rows: int, order, stream=None):
    """``order``: device memory of at least zero_token_order_bytes bytes, of any type."""
    dev = _device()
    ids, n = _tokens(tokens, dev)
    p, nbytes = _memory(order, "order", dev)
    _fits(rows, "rows")
    rc = _lib.zero_token_order(ids, _IDS[tokens.dtype], n, rows, p, nbytes, _stream(stream, dev))
    if rc:
        zero._check("zero_token_order", rc)


def zero_embedding_grad_workspace_bytes(n: int, dim: int) -> int:
    return _sized("zero_embedding_grad_workspace_bytes", n, dim)


def zero_embedding_grad(order, rows: int, d_out, grad, workspace, scale: float = 1.0, first: int = 0,
                        accumulate: bool = False, stream=None):
    """``d_out`` [number of tokens, dim], in the tokens' order; ``grad``: the
    elements of the flat [rows, dim] gradient from ``first`` on, as many as it has
    (the whole table's by default)."""
    dev = _device()
    src, stride = _rows(d_out, "d_out", dev, None, _TYPES)
    n, dim = d_out.shape
    p, order_bytes = _memory(order, "order", dev)
    _fits(rows, "rows")
    _fits(first, "first")
    need = _lib.zero_token_order_bytes(n, rows)
    if order_bytes < need:
        raise ValueError(f"order: {order_bytes} bytes given, the call reaches {need}")
    ws, ws_bytes = _memory(workspace, "workspace", dev)
    count = grad.numel() if hasattr(grad, "numel") else 0
    dst = _flat(grad, "grad", dev, count, _TYPES)
    rc = _lib.zero_embedding_grad(p, n, rows, dim, src, _TYPES[d_out.dtype], stride, scale, dst, _TYPES[grad.dtype],
                                  first, count, 1 if accumulate else 0, ws, ws_bytes, _stream(stream, dev))
    if rc:
        zero._check("zero_embedding_grad", rc)


def _vectors(dev, dim, a, a_name, b, b_name):
    """Addresses of two vectors, either of which may be missing, and the type that they share."""
    if a is None:
        if b is None:
            return 0, 0, ZERO_F32
        return 0, _flat(b, b_name, dev, dim, _TYPES), _TYPES[b.dtype]
    pa = _flat(a, a_name, dev, dim, _TYPES)
    kind = a.dtype
    return pa, 0 if b is None else _flat(b, b_name, dev, dim, (kind,)), _TYPES[kind]


# zero_norm_args and zero_norm_grad_args as bytes: a third of the time of a ctypes structure
_NORM = struct.Struct("8Q6qd4i")
_NORM_GRAD = struct.Struct("9Q6q6i")


def zero_norm(x, y, mean=None, rstd=None, weight=None, bias=None, eps: float = 1e-5, residual=None, total=None,
              rms: bool = False, stream=None):
    """``y`` = the norm of the rows of ``x`` [n, dim], or of ``total`` = x +
    ``residual``; ``mean`` and ``rstd`` [n], float32, for the backward pass.
    ``rms``: without the mean."""
    dev = _device()
    px, sx = _rows(x, "x", dev, None, _TYPES)
    size, kind = x.shape, x.dtype
    (n, dim), kinds = size, (kind,)
    py, sy = _rows(y, "y", dev, size, kinds)
    if (residual is None) != (total is None):
        raise ValueError("residual and total: both or neither")
    pr = pt = sr = st = 0
    if total is not None:
        pr, sr = _rows(residual, "residual", dev, size, kinds)
        pt, st = _rows(total, "total", dev, size, kinds)
    pw, pb, w_type = _vectors(dev, dim, weight, "weight", bias, "bias")
    pm = 0 if mean is None else _flat(mean, "mean", dev, n, _F32)
    ps = 0 if rstd is None else _flat(rstd, "rstd", dev, n, _F32)
    rc = _lib.zero_norm(_NORM.pack(px, pr, pt, py, pw, pb, pm, ps, n, dim, sx, sr, st, sy, eps, _TYPES[kind], w_type,
                                   1 if rms else 0, 0), _stream(stream, dev))
    if rc:
        zero._check("zero_norm", rc)


def zero_norm_grad_workspace_bytes(n: int, dim: int) -> int:
    return _sized("zero_norm_grad_workspace_bytes", n, dim)


def zero_norm_grad(d_y, x, mean, rstd, d_x=None, workspace=None, weight=None, d_weight=None, d_bias=None, d_total=None,
                   accumulate: bool = False, rms: bool = False, stream=None):
    """The gradient of zero_norm. ``x``: what was normalised (``total`` where a
    residual was added); ``d_total``: the gradient that reaches it by the skip path;
    ``d_x``: of x and of the residual alike. ``accumulate``: add to ``d_weight``
    and ``d_bias``."""
    dev = _device()
    px, sx = _rows(x, "x", dev, None, _TYPES)
    size, kind = x.shape, x.dtype
    (n, dim), kinds = size, (kind,)
    py, sy = _rows(d_y, "d_y", dev, size, kinds)
    pt = st = pd = sd = ws = ws_bytes = pm = 0
    if d_total is not None:
        pt, st = _rows(d_total, "d_total", dev, size, kinds)
    if d_x is not None:
        pd, sd = _rows(d_x, "d_x", dev, size, kinds)
    pw, _, w_type = _vectors(dev, dim, weight, "weight", None, "")
    pgw, pgb, g_type = _vectors(dev, dim, d_weight, "d_weight", d_bias, "d_bias")
    if not rms:
        pm = _flat(mean, "mean", dev, n, _F32)
    ps = _flat(rstd, "rstd", dev, n, _F32)
    if workspace is not None:
        ws, ws_bytes = _memory(workspace, "workspace", dev)
    rc = _lib.zero_norm_grad(_NORM_GRAD.pack(py, px, pt, pd, pw, pm, ps, pgw, pgb, n, dim, sy, sx, st, sd, _TYPES[kind],
                                             w_type, g_type, 1 if rms else 0, 1 if accumulate else 0, 0),
                             ws, ws_bytes, _stream(stream, dev))
    if rc:
        zero._check("zero_norm_grad", rc)
