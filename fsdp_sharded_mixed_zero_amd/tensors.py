"""Python binding of the tensor-list calls of libzero_mi355x.so, declared in
include/zero_tensors.h: the same names, argument marshalling only.

A list is described once (``zero_tensors``: parameters, fp32 masters, moments,
groups), which also writes its device table; a step then passes the gradients,
as a list of tensors (None: no gradient this time) or, made once, as
``zero.pointer_array(grads)``. Conventions, streams and errors are those of
``zero``. Lists of tensors are checked (device, type, length, contiguity)
before a call; a pointer array, like a raw address, is the caller's to get
right, apart from the alignment and overlap that the library itself checks.
"""

from __future__ import annotations

import ctypes

from . import zero

ZERO_BF16 = 0
ZERO_F32 = 1
ZERO_STATE8_BLOCK = 256         # elements of a tensor that share one scale (include/zero_tensors.h)
ZERO_TENSOR_GROUPS = 8
ZERO_TENSORS_PER_LAUNCH = 768   # tensors one launch carries


class zero_tensor(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("master", ctypes.c_void_p), ("m", ctypes.c_void_p),
                ("v", ctypes.c_void_p), ("m_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("len", ctypes.c_int64), ("group", ctypes.c_int32), ("reserved", ctypes.c_int32)]


_VP = ctypes.c_void_p
_I32 = ctypes.c_int32
_PP = _VP     # host arrays of pointers (ctypes passes an array as its address)

_SIGNATURES = {
    "zero_tensors": (ctypes.c_int, [ctypes.POINTER(zero_tensor), _I32, _I32, _I32, _I32, ctypes.POINTER(_VP)]),
    "zero_tensors_free": (None, [_VP]),
    "zero_tensors_table_bytes": (ctypes.c_size_t, [_VP]),
    "zero_tensors_upload": (ctypes.c_int, [_VP, _VP, ctypes.c_size_t, _VP]),
    "zero_tensors_sqnorm_workspace_bytes": (ctypes.c_size_t, [_VP]),
    "zero_tensors_sqnorm": (ctypes.c_int, [_VP, _PP, _VP, _I32, _VP, ctypes.c_size_t, _VP]),
    "zero_tensors_adamw_step": (ctypes.c_int, [_VP, _PP, _VP, _I32, _VP, _I32,
                                               _VP]),
    "zero_tensors_state_import": (ctypes.c_int, [_VP, _PP, _PP, _VP]),
    "zero_tensors_state_export": (ctypes.c_int, [_VP, _PP, _PP, _VP]),
}

_lib = None


def library():
    """The library's handle with the tensor-list calls' signatures set."""
    global _lib
    if _lib is None:
        lib = zero.library()
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def state8_blocks(n: int) -> int:
    """Scales that a tensor of n elements needs for each of its 8-bit moments."""
    return -(-int(n) // ZERO_STATE8_BLOCK)


_torch_c = None


def _stream(stream):
    """The stream's handle, as zero._stream gives it; the current stream's by
    the short way (0.1 us against 2.6 us for the stream object, of a call that
    takes 6)."""
    global _torch_c
    if stream is not None:
        return zero._stream(stream)
    if _torch_c is None:
        from torch import _C
        _torch_c = _C
    return _torch_c._cuda_getCurrentRawStream(_torch_c._cuda_getDevice())


def _call(name, lst, stream, *args):
    """One call of the library on the list. The list's table is marked as in
    use on the stream, so that its memory, freed with the list, is not given
    out before the work is done."""
    stream = _stream(stream)
    rc = getattr(_lib or library(), name)(lst.handle, *args, stream)
    if rc:
        zero._check(name, rc)
    if stream not in lst._streams:
        lst._use(stream)


def _type_of(dtype, what):
    import torch
    if dtype == torch.bfloat16:
        return ZERO_BF16
    if dtype == torch.float32:
        return ZERO_F32
    raise TypeError(f"{what}: bfloat16 or float32 expected, got {dtype}")


def _check(tensors, lens, dtypes, device, what):
    """Refuse a list of tensors that the list's lengths, types or device do not fit."""
    if len(tensors) != len(lens):
        raise ValueError(f"{what}: {len(tensors)} entries for a list of {len(lens)} tensors")
    for i, (t, n) in enumerate(zip(tensors, lens)):
        if t is None:
            continue
        if not getattr(t, "is_cuda", False):
            raise TypeError(f"{what} {i}: device memory expected, got {type(t).__name__}")
        if t.dtype not in dtypes:
            raise TypeError(f"{what} {i}: {' or '.join(str(d) for d in dtypes)} expected, got {t.dtype}")
        if t.device != device:
            raise ValueError(f"{what} {i} is on {t.device}, the list on {device}")
        if t.numel() != n:
            raise ValueError(f"{what} {i}: {t.numel()} elements, the list's tensor has {n}")
        if not t.is_contiguous():
            raise ValueError(f"{what} {i}: a contiguous tensor is expected")


class TensorList:
    """Owner of a zero_tensors_t handle and of its device table; keeps the
    tensors it was made from."""

    def __init__(self, handle, lens, grad_dtype, state_bits, device, table, keep):
        self.handle = handle
        self.lens = lens
        self.n_tensors = len(lens)
        self.grad_dtype = grad_dtype
        self.state_bits = state_bits
        self.device = device
        self.table = table
        self._keep = keep
        self._streams = set()

    def _use(self, handle):
        import torch
        self._streams.add(handle)
        if isinstance(self.table, int):     # memory that the caller keeps
            return
        self.table.record_stream(torch.cuda.ExternalStream(handle, device=self.device))

    def close(self):
        if self.handle:
            library().zero_tensors_free(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def zero_tensors(param, m, v, master=None, m_scale=None, v_scale=None, group=None, grad_dtype=None,
                 stream=None) -> TensorList:
    """Describe a list and write its table. ``param``: bfloat16 tensors, with
    float32 ``master`` tensors, or float32 ones without. ``m``, ``v``: float32
    tensors, or one byte per element (float8_e4m3fn, uint8 or int8) with
    float32 scales, ``state8_blocks`` of them per tensor (for a beta2 of up to
    0.95: beyond, the 8-bit second moment does not follow its gradients over
    many steps). ``group``: one index per tensor (default 0). ``grad_dtype``:
    the gradients' type (default: the parameters'). The call waits until the table is written, unless a stream
    is being captured: then the graph's replays write it, and a call outside
    the graph reads it only after one of them."""
    import torch

    param = list(param)
    if not param:
        raise ValueError("a list of at least one tensor is expected")
    lens = [int(t.numel()) for t in param]
    device = param[0].device
    p_type = _type_of(param[0].dtype, "param")
    grad_dtype = param[0].dtype if grad_dtype is None else grad_dtype
    g_type = _type_of(grad_dtype, "grad_dtype")
    first = next((t for t in m if t is not None), None)    # None: only tensors without elements
    bits = 8 if first is not None and first.dtype != torch.float32 else 32
    state = (torch.float32,) if bits == 32 else (torch.float8_e4m3fn, torch.uint8, torch.int8)
    blocks = [state8_blocks(n) for n in lens]
    f32 = (torch.float32,)
    columns = [("param", param, lens, (param[0].dtype,)), ("master", master, lens, f32), ("m", m, lens, state),
               ("v", v, lens, state), ("m_scale", m_scale, blocks, f32), ("v_scale", v_scale, blocks, f32)]
    arr = (zero_tensor * len(lens))()
    for name, tensors, sizes, dtypes in columns:
        if tensors is None:
            continue
        _check(tensors, sizes, dtypes, device, name)
        for rec, t, n in zip(arr, tensors, lens):
            setattr(rec, name, t.data_ptr() if t is not None and n else None)
    if group is not None and len(group) != len(lens):
        raise ValueError(f"group: {len(group)} entries for a list of {len(lens)} tensors")
    for i, (rec, n) in enumerate(zip(arr, lens)):
        k = int(group[i]) if group is not None else 0
        if not -(1 << 31) <= k < 1 << 31:       # the record would hold another one
            raise ValueError(f"group {k} of tensor {i} outside [0, {ZERO_TENSOR_GROUPS})")
        rec.len, rec.group = n, k
    h = _VP()
    zero._check("zero_tensors", library().zero_tensors(arr, len(lens), p_type, g_type, bits, ctypes.byref(h)))
    lst = TensorList(h.value, lens, grad_dtype, bits, device, None,
                     [list(c) for _, c, _, _ in columns if c is not None])
    with torch.cuda.device(device):
        nbytes = library().zero_tensors_table_bytes(h)
        capturing = torch.cuda.is_current_stream_capturing()
        # the table's memory belongs to the stream that writes it: memory that another stream
        # has freed may still be written by that stream's pending work
        with torch.cuda.stream(torch.cuda.ExternalStream(_stream(stream), device=device)):
            lst.table = torch.empty((nbytes + 7) // 8, dtype=torch.int64, device=device)
            _call("zero_tensors_upload", lst, stream, lst.table.data_ptr(), nbytes)
            capturing = capturing or torch.cuda.is_current_stream_capturing()
        if not capturing:
            torch.cuda.synchronize(device)
    return lst


def zero_tensors_free(lst: TensorList) -> None:
    lst.close()


def zero_tensors_table_bytes(lst: TensorList) -> int:
    return int(library().zero_tensors_table_bytes(lst.handle))


def zero_tensors_upload(lst: TensorList, table, table_bytes: int | None = None, stream=None) -> None:
    """Write the list's table into ``table`` and bind the list to it. The table
    before (``lst.table``) has to be kept as long as a graph captured with it
    may be replayed."""
    if table_bytes is None:
        table_bytes = table.numel() * table.element_size()
    zero._need(table, table_bytes, "table")
    handle = _stream(stream)
    zero._check("zero_tensors_upload", library().zero_tensors_upload(lst.handle, zero._ptr(table), table_bytes, handle))
    lst.table, lst._streams = table, set()
    lst._use(handle)


def zero_tensors_sqnorm_workspace_bytes(lst: TensorList) -> int:
    return int(library().zero_tensors_sqnorm_workspace_bytes(lst.handle))


def _pointers(lst, tensors, dtype, what):
    """``dtype`` None: float32."""
    if not isinstance(tensors, ctypes.Array):
        if dtype is None:
            from torch import float32 as dtype
        _check(tensors, lst.lens, (dtype,), lst.device, what)
        return zero._ptr_array([t if n else None for t, n in zip(tensors, lst.lens)])
    if len(tensors) < lst.n_tensors:
        raise ValueError(f"{what}: {len(tensors)} pointers for a list of {lst.n_tensors} tensors")
    return tensors


def zero_tensors_sqnorm(lst: TensorList, tensor_grads, out, accumulate: bool, workspace, ws_bytes: int | None = None,
                        stream=None):
    arr = _pointers(lst, tensor_grads, lst.grad_dtype, "gradient")
    zero._need(out, 8, "output")
    if ws_bytes is None:
        ws_bytes = workspace.numel() * workspace.element_size()
    else:
        zero._need(workspace, ws_bytes, "workspace")
    _call("zero_tensors_sqnorm", lst, stream, arr, zero._ptr(out), 1 if accumulate else 0, zero._ptr(workspace),
          ws_bytes)


def group_array(hp):
    """The hyperparameters of a step's groups: one zero.hparams, or a list."""
    if isinstance(hp, ctypes.Array):
        return hp
    hp = [hp] if isinstance(hp, zero.zero_adamw_hparams) else list(hp)
    return (zero.zero_adamw_hparams * len(hp))(*hp)


def zero_tensors_adamw_step(lst: TensorList, tensor_grads, hp, rank_sqnorms, n_ranks: int, stream=None):
    """``hp``: one zero.hparams, or a list of them, one per group. With an 8-bit
    state, beta2 up to 0.95 (include/zero_tensors.h, "Over many steps")."""
    arr = _pointers(lst, tensor_grads, lst.grad_dtype, "gradient")
    groups = group_array(hp)
    if n_ranks > 0:
        zero._need(rank_sqnorms, 8 * n_ranks, "rank sums of squares")
    _call("zero_tensors_adamw_step", lst, stream, arr, groups, len(groups), zero._ptr(rank_sqnorms), n_ranks)


def _state8(name, lst, m, v, stream):
    _call(name, lst, stream, _pointers(lst, m, None, "m"), _pointers(lst, v, None, "v"))


def zero_tensors_state_import(lst: TensorList, m, v, stream=None):
    _state8("zero_tensors_state_import", lst, m, v, stream)


def zero_tensors_state_export(lst: TensorList, m, v, stream=None):
    _state8("zero_tensors_state_export", lst, m, v, stream)
