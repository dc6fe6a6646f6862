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

from . import tensors, zero
from .tensors import ZERO_BF16, ZERO_F32  # noqa: F401 (the types of a call's arrays)

ZERO_I32 = 2
ZERO_I64 = 3
ZERO_LAYER_ROWS = 16777215
ZERO_LAYER_DIM = 1048576
ZERO_LAYER_ELEMS = 34359738368
ZERO_EMBEDDING_PIECE = 32

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
    "zero_norm": (ctypes.c_int, [ctypes.POINTER(zero_norm_args), _VP]),
    "zero_norm_grad_workspace_bytes": (ctypes.c_size_t, [_I64, _I64]),
    "zero_norm_grad": (ctypes.c_int, [ctypes.POINTER(zero_norm_grad_args), _VP, ctypes.c_size_t, _VP]),
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


def _call(name, stream, *args):
    rc = getattr(_lib or library(), name)(*args, tensors._stream(stream))
    if rc:
        zero._check(name, rc)


def _sized(name, *sizes):
    """Bytes of an order or a workspace."""
    nbytes = int(getattr(_lib or library(), name)(*sizes))
    if nbytes == 0:
        raise ValueError(f"{name}: sizes {sizes} outside the limits of include/zero_layers.h")
    return nbytes


class _Device:
    """The device that a call's tensors share: the current one."""

    def __init__(self):
        import torch
        self.torch = torch
        self.at = torch.cuda.current_device() if torch.cuda.is_available() else None

    def check(self, t, what):
        if not getattr(t, "is_cuda", False):
            raise TypeError(f"{what}: device memory expected, got {type(t).__name__}")
        if t.device.index != self.at:
            raise ValueError(f"{what} is on {t.device}, the current device is {self.at}")

    def rows(self, t, what, shape=None, dtype=None):
        """Address and stride of an array of rows."""
        self.check(t, what)
        if t.dim() != 2 or (shape is not None and tuple(t.shape) != tuple(shape)):
            raise ValueError(f"{what}: {'two dimensions' if shape is None else tuple(shape)} expected, got "
                             f"{tuple(t.shape)}")
        if dtype is not None and t.dtype != dtype:
            raise TypeError(f"{what}: {dtype} expected, got {t.dtype}")
        n, dim = t.shape
        if dim > 1 and t.stride(1) != 1:
            raise ValueError(f"{what}: the elements of a row have to be consecutive")
        return t.data_ptr() if t.numel() else None, int(t.stride(0)) if n > 1 else int(dim)

    def flat(self, t, what, count, dtypes):
        """Address of an array without gaps of `count` elements (None: as many as it has)."""
        self.check(t, what)
        if t.dtype not in dtypes:
            raise TypeError(f"{what}: {' or '.join(str(d) for d in dtypes)} expected, got {t.dtype}")
        if count is not None and t.numel() != count:
            raise ValueError(f"{what}: {t.numel()} elements, {count} expected")
        if not t.is_contiguous():
            raise ValueError(f"{what}: a contiguous tensor is expected")
        return t.data_ptr() if t.numel() else None

    def memory(self, t, what):
        """Address and bytes of an order or a workspace."""
        self.check(t, what)
        if not t.is_contiguous():
            raise ValueError(f"{what}: a contiguous tensor is expected")
        return t.data_ptr(), t.numel() * t.element_size()

    def tokens(self, t):
        torch = self.torch
        p = self.flat(t, "tokens", None, (torch.int32, torch.int64))
        return p, ZERO_I32 if t.dtype == torch.int32 else ZERO_I64, t.numel()


def _type(t, what):
    return tensors._type_of(t.dtype, what)


def zero_embedding(tokens, table, out, scale: float = 1.0, stream=None):
    """``out`` [number of tokens, dim] = scale * rows of ``table`` [rows, dim]."""
    dev = _Device()
    ids, id_type, n = dev.tokens(tokens)
    src, _ = dev.rows(table, "table")
    if not table.is_contiguous():
        raise ValueError("table: a contiguous tensor is expected")
    rows, dim = table.shape
    dst, stride = dev.rows(out, "out", (n, dim))
    _call("zero_embedding", stream, ids, id_type, n, src, _type(table, "table"), rows, dim, scale, dst,
          _type(out, "out"), stride)


def zero_token_order_bytes(n: int, rows: int) -> int:
    return _sized("zero_token_order_bytes", n, rows)


def zero_token_order(tokens, rows: int, order, stream=None):
    """``order``: device memory of at least zero_token_order_bytes bytes, of any type."""
    dev = _Device()
    ids, id_type, n = dev.tokens(tokens)
    p, nbytes = dev.memory(order, "order")
    _call("zero_token_order", stream, ids, id_type, n, rows, p, nbytes)


def zero_embedding_grad_workspace_bytes(n: int, dim: int) -> int:
    return _sized("zero_embedding_grad_workspace_bytes", n, dim)


def zero_embedding_grad(order, rows: int, d_out, grad, workspace, scale: float = 1.0, first: int = 0,
                        accumulate: bool = False, stream=None):
    """``d_out`` [number of tokens, dim], in the tokens' order; ``grad``: the
    elements of the flat [rows, dim] gradient from ``first`` on, as many as it has
    (the whole table's by default)."""
    dev = _Device()
    src, stride = dev.rows(d_out, "d_out")
    n, dim = d_out.shape
    p, order_bytes = dev.memory(order, "order")
    zero._need(order, zero_token_order_bytes(n, rows), "order")
    ws, ws_bytes = dev.memory(workspace, "workspace")
    dst = dev.flat(grad, "grad", None, (dev.torch.bfloat16, dev.torch.float32))
    _call("zero_embedding_grad", stream, p, n, rows, dim, src, _type(d_out, "d_out"), stride, scale, dst,
          _type(grad, "grad"), first, grad.numel(), 1 if accumulate else 0, ws, ws_bytes)


def _vectors(dev, dim, pairs):
    """Addresses of the vectors that are there, which share one type, and that type."""
    kind, at = None, {}
    for name, t in pairs.items():
        if t is None:
            continue
        at[name] = dev.flat(t, name, dim, (dev.torch.bfloat16, dev.torch.float32) if kind is None else (kind,))
        kind = t.dtype
    return at, ZERO_F32 if kind is None or kind == dev.torch.float32 else ZERO_BF16


def zero_norm(x, y, mean=None, rstd=None, weight=None, bias=None, eps: float = 1e-5, residual=None, total=None,
              rms: bool = False, stream=None):
    """``y`` = the norm of the rows of ``x`` [n, dim], or of ``total`` = x +
    ``residual``; ``mean`` and ``rstd`` [n], float32, for the backward pass.
    ``rms``: without the mean."""
    dev = _Device()
    n, dim = x.shape if x.dim() == 2 else (0, 0)
    a = zero_norm_args(n=n, dim=dim, eps=eps, type=_type(x, "x"), rms=1 if rms else 0)
    for name, t in (("x", x), ("y", y), ("residual", residual), ("total", total)):
        if t is not None:
            p, stride = dev.rows(t, name, None if t is x else (n, dim), x.dtype)
            setattr(a, name, p)
            setattr(a, name + "_stride", stride)
    if (residual is None) != (total is None):
        raise ValueError("residual and total: both or neither")
    at, a.weight_type = _vectors(dev, dim, {"weight": weight, "bias": bias})
    for name, p in at.items():
        setattr(a, name, p)
    for name, t in (("mean", mean), ("rstd", rstd)):
        if t is not None:
            setattr(a, name, dev.flat(t, name, n, (dev.torch.float32,)))
    _call("zero_norm", stream, ctypes.byref(a))


def zero_norm_grad_workspace_bytes(n: int, dim: int) -> int:
    return _sized("zero_norm_grad_workspace_bytes", n, dim)


def zero_norm_grad(d_y, x, mean, rstd, d_x=None, workspace=None, weight=None, d_weight=None, d_bias=None, d_total=None,
                   accumulate: bool = False, rms: bool = False, stream=None):
    """The gradient of zero_norm. ``x``: what was normalised (``total`` where a
    residual was added); ``d_total``: the gradient that reaches it by the skip path;
    ``d_x``: of x and of the residual alike. ``accumulate``: add to ``d_weight``
    and ``d_bias``."""
    dev = _Device()
    n, dim = x.shape if x.dim() == 2 else (0, 0)
    a = zero_norm_grad_args(n=n, dim=dim, type=_type(x, "x"), rms=1 if rms else 0, accumulate=1 if accumulate else 0)
    for name, t in (("x", x), ("d_y", d_y), ("d_total", d_total), ("d_x", d_x)):
        if t is not None:
            p, stride = dev.rows(t, name, None if t is x else (n, dim), x.dtype)
            setattr(a, name, p)
            setattr(a, name + "_stride", stride)
    at, a.weight_type = _vectors(dev, dim, {"weight": weight})
    more, a.grad_type = _vectors(dev, dim, {"d_weight": d_weight, "d_bias": d_bias})
    for name, p in {**at, **more}.items():
        setattr(a, name, p)
    for name, t in (("mean", None if rms else mean), ("rstd", rstd)):
        if t is not None:
            setattr(a, name, dev.flat(t, name, n, (dev.torch.float32,)))
    ws, ws_bytes = (None, 0) if workspace is None else dev.memory(workspace, "workspace")
    _call("zero_norm_grad", stream, ctypes.byref(a), ws, ws_bytes)
