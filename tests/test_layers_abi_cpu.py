"""The token-table and norm calls on the host: every declared symbol is exported
and bound, constants and records agree with the header, and every refusal that
the header names is made before anything is enqueued. Addresses are made up: no
call here reaches a launch."""

import ctypes
import os
import re

import pytest

from fsdp_sharded_mixed_zero_amd import layers, zero

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "zero_layers.h")

pytestmark = pytest.mark.skipif(not os.path.exists(zero.LIB_PATH),
                                reason="libzero_mi355x.so not built (run __graft_entry__.build())")

BASE, FAR = 1 << 40, 1 << 34
BF16, F32, I32, I64 = layers.ZERO_BF16, layers.ZERO_F32, layers.ZERO_I32, layers.ZERO_I64


def at(k):
    """A made-up address, far from every other one."""
    return BASE + k * FAR


def header():
    return re.sub(r"/\*.*?\*/", "", open(HEADER, encoding="utf-8").read(), flags=re.S)


def refused(rc, text):
    assert rc == zero.ZERO_EINVAL, rc
    assert text in zero.zero_last_error(), zero.zero_last_error()


def test_declared_symbols_are_exported_and_bound():
    names = sorted(set(re.findall(r"\b(zero_[a-z0-9_]*)\s*\(", header())))
    assert len(names) == 8, names
    for name in names:
        assert hasattr(layers.library(), name)
        assert callable(getattr(layers, name))
    assert set(names) == set(layers._SIGNATURES)


def test_constants_and_records_agree_with_the_header():
    text = header()
    for name in ("ZERO_I32", "ZERO_I64", "ZERO_LAYER_ROWS", "ZERO_LAYER_DIM", "ZERO_LAYER_ELEMS"):
        assert int(re.search(rf"#define {name} (\d+)", text)[1]) == getattr(layers, name), name
    for record, packed in ((layers.zero_norm_args, layers._NORM), (layers.zero_norm_grad_args, layers._NORM_GRAD)):
        body = re.search(rf"typedef struct \{{([^}}]*)\}} {record.__name__};", text, re.S)[1]
        fields = [f for line in re.findall(r"[^;]+;", body) for f in re.findall(r"(\w+)\s*[,;]", line)]
        assert fields == [f for f, _ in record._fields_]
        assert ctypes.sizeof(record) == packed.size
        sizes = {"Q": 8, "q": 8, "d": 8, "i": 4}
        kinds = [c for n, c in re.findall(r"(\d*)([Qqdi])", packed.format) for _ in range(int(n or 1))]
        assert [sizes[c] for c in kinds] == [ctypes.sizeof(t) for _, t in record._fields_]


def embedding(**over):
    a = dict(tokens=at(0), token_type=I64, n=10, table=at(1), table_type=BF16, rows=100, dim=8, scale=1.0, out=at(2),
             out_type=BF16, stride=8)
    a.update(over)
    return layers.library().zero_embedding(*a.values(), None)


@pytest.mark.parametrize("over,text", [
    (dict(token_type=BF16), "token type"), (dict(table_type=I32), "element type"), (dict(out_type=7), "element type"),
    (dict(n=-1), "n ="), (dict(n=layers.ZERO_LAYER_ROWS + 1), "n ="), (dict(rows=0), "rows ="),
    (dict(rows=layers.ZERO_LAYER_ROWS + 1), "rows ="), (dict(dim=0), "dim ="),
    (dict(dim=layers.ZERO_LAYER_DIM + 1), "dim ="), (dict(n=1 << 20, dim=1 << 16, stride=1 << 16), "2^35"),
    (dict(scale=float("nan")), "scale"), (dict(scale=1e39), "scale"), (dict(scale=float("-inf")), "scale"),
    (dict(tokens=None), "tokens is NULL"), (dict(table=None), "table is NULL"), (dict(out=None), "out is NULL"),
    (dict(tokens=at(0) + 4), "misaligned"), (dict(table=at(1) + 1), "misaligned"),
    (dict(out_type=F32, out=at(2) + 2), "misaligned"), (dict(stride=7), "stride"), (dict(stride=-8), "stride"),
    (dict(out=at(1) + 16), "overlaps"), (dict(out=at(0) + 16), "overlaps"), (dict(tokens=at(2) + 144), "overlaps"),
])
def test_embedding_refusals(over, text):
    refused(embedding(**over), text)


def test_no_tokens_need_no_arrays():
    assert embedding(n=0, tokens=None, table=None, out=None, stride=0) == 0


def order_call(**over):
    a = dict(tokens=at(0), token_type=I32, n=100, rows=50, order=at(1), nbytes=1 << 20)
    a.update(over)
    return layers.library().zero_token_order(*a.values(), None)


@pytest.mark.parametrize("over,text", [
    (dict(token_type=0), "token type"), (dict(n=-5), "n ="), (dict(n=1 << 24), "n ="), (dict(rows=0), "rows ="),
    (dict(order=None), "NULL"), (dict(order=at(1) + 8), "16-byte"), (dict(nbytes=64), "need"),
    (dict(tokens=None), "tokens is NULL"), (dict(tokens=at(0) + 2), "misaligned"), (dict(tokens=at(1) + 400), "overlaps"),
])
def test_order_refusals(over, text):
    refused(order_call(**over), text)


def test_bytes_grow_with_the_batch_and_are_zero_outside_the_limits():
    lib = layers.library()
    ns = [0, 1, 7, 8, 100, 4095, 4096, 4097, 5000, 8191, 12288, 12289, 20000, 1 << 20, layers.ZERO_LAYER_ROWS]
    for sizes in ([lib.zero_token_order_bytes(n, 50257) for n in ns],
                  [lib.zero_embedding_grad_workspace_bytes(n, 777) for n in ns],
                  [lib.zero_norm_grad_workspace_bytes(n, 777) for n in ns],
                  [lib.zero_norm_grad_workspace_bytes(n, 20000) for n in ns[:-2]]):
        assert all(a <= b for a, b in zip(sizes, sizes[1:])) and sizes[0] > 0 and all(b % 4 == 0 for b in sizes)
    for name in ("zero_token_order_bytes", "zero_embedding_grad_workspace_bytes", "zero_norm_grad_workspace_bytes"):
        for bad in ((-1, 5), (1 << 24, 5), (5, 0), (5, (1 << 24) if "order" in name else (1 << 20) + 1)):
            assert getattr(lib, name)(*bad) == 0
            with pytest.raises(ValueError, match="limits"):
                getattr(layers, name)(*bad)


def grad_call(**over):
    a = dict(order=at(0), n=100, rows=50, dim=8, d_out=at(1), out_type=BF16, stride=8, scale=1.0, grad=at(2),
             grad_type=F32, first=0, count=400, accumulate=0, ws=at(3), ws_bytes=1 << 20)
    a.update(over)
    return layers.library().zero_embedding_grad(*a.values(), None)


@pytest.mark.parametrize("over,text", [
    (dict(out_type=I64), "element type"), (dict(grad_type=-1), "element type"), (dict(n=-1), "n ="),
    (dict(rows=1 << 24), "rows ="), (dict(dim=0), "dim ="), (dict(scale=float("inf")), "scale"),
    (dict(first=-1), "a table of 400"), (dict(count=-1), "a table of 400"), (dict(first=1), "a table of 400"),
    (dict(first=401, count=0), "a table of 400"), (dict(rows=1 << 22, dim=1 << 14, stride=1 << 14, count=(1 << 35) + 1), "2^35"), (dict(first=1 << 62, count=1 << 62), "a table of 400"),
    (dict(order=None), "NULL order"), (dict(ws=None), "NULL order or workspace"), (dict(ws=at(3) + 4), "16-byte"),
    (dict(order=at(0) + 4), "16-byte"), (dict(ws_bytes=16), "need"), (dict(d_out=None), "d_out is NULL"),
    (dict(grad=None), "grad is NULL"), (dict(grad=at(2) + 2), "misaligned"), (dict(d_out=at(1) + 1), "misaligned"),
    (dict(stride=-1), "stride"), (dict(grad=at(0) + 64), "overlaps"), (dict(grad=at(1) + 4), "overlaps"),
    (dict(ws=at(1) + 16), "overlaps"), (dict(ws=at(2) + 16), "overlaps"), (dict(ws=at(0) + 16), "overlaps"),
])
def test_table_gradient_refusals(over, text):
    refused(grad_call(**over), text)


def test_an_empty_part_is_nothing_to_do():
    assert grad_call(first=400, count=0, grad=None) == 0
    assert grad_call(first=3, count=0, grad=None) == 0


def norm_call(**over):
    a = dict(x=at(0), residual=None, total=None, y=at(1), weight=at(2), bias=at(3), mean=at(4), rstd=at(5), n=10, dim=16,
             x_stride=16, residual_stride=16, total_stride=16, y_stride=16, eps=1e-5, type=BF16, weight_type=F32)
    a.update(over)
    return layers.library().zero_norm(ctypes.byref(layers.zero_norm_args(**a)), None)


@pytest.mark.parametrize("over,text", [
    (dict(type=I32), "element type"), (dict(weight_type=9), "element type"), (dict(n=-1), "n ="), (dict(dim=0), "dim ="),
    (dict(dim=(1 << 20) + 1), "dim ="), (dict(eps=-1e-9), "eps"), (dict(eps=float("nan")), "eps"), (dict(eps=1e39), "eps"),
    (dict(total=at(6)), "residual and total"), (dict(residual=at(6)), "residual and total"), (dict(x=None), "x is NULL"),
    (dict(y=None), "y is NULL"), (dict(x=at(0) + 1), "misaligned"), (dict(weight=at(2) + 2), "misaligned"),
    (dict(rstd=at(5) + 2), "misaligned"), (dict(y_stride=15), "stride"), (dict(x_stride=-16), "stride"),
    (dict(y=at(0) + 32), "overlaps"), (dict(y=at(0), y_stride=32), "overlaps"), (dict(y=at(2)), "overlaps"),
    (dict(mean=at(1) + 4), "overlaps"), (dict(mean=at(5)), "overlaps"),
    (dict(residual=at(6), total=at(1)), "overlaps"), (dict(residual=at(6), total=at(0), y=at(0)), "overlaps"),
    (dict(residual=at(6), total=at(7), y=at(6)), "overlaps"), (dict(residual=at(6), total=at(6) + 2), "overlaps"),
])
def test_norm_refusals(over, text):
    refused(norm_call(**over), text)


def test_columns_of_one_array_do_not_overlap():
    """x and y as halves of one array's rows: their ranges meet, their elements do not. Refused for another reason
    (the weight), so that nothing is launched; one column more and they do overlap."""
    weight = dict(weight=at(2) + 1)
    halves = dict(x=at(0), y=at(0) + 32, x_stride=32, y_stride=32)
    refused(norm_call(**halves, **weight), "weight is misaligned")
    refused(norm_call(**{**halves, "y": at(0) + 30}), "overlaps")
    refused(norm_call(**{**halves, "y": at(0) + 34}), "overlaps")        # into the next row's x
    refused(norm_call(**{**halves, "y": at(0) + 32 + 64 * 3, "mean": at(0) + 32}), "overlaps")


def norm_grad_call(ws=at(20), ws_bytes=1 << 24, **over):
    a = dict(d_y=at(0), x=at(1), d_total=at(2), d_x=at(3), weight=at(4), mean=at(5), rstd=at(6), d_weight=at(7),
             d_bias=at(8), n=10, dim=16, d_y_stride=16, x_stride=16, d_total_stride=16, d_x_stride=16, type=BF16,
             weight_type=BF16, grad_type=F32)
    a.update(over)
    return layers.library().zero_norm_grad(ctypes.byref(layers.zero_norm_grad_args(**a)), ws, ws_bytes, None)


@pytest.mark.parametrize("over,text", [
    (dict(type=I32), "element type"), (dict(weight_type=3), "element type"), (dict(grad_type=3), "element type"),
    (dict(n=1 << 24), "n ="), (dict(dim=0), "dim ="), (dict(d_x=None, d_weight=None, d_bias=None), "no output"),
    (dict(d_x=None), "d_total without d_x"), (dict(ws=None), "NULL workspace"), (dict(ws=at(20) + 4), "16-byte"),
    (dict(ws_bytes=127), "need"), (dict(d_y=None), "d_y is NULL"), (dict(x=None), "x is NULL"),
    (dict(mean=None), "mean is NULL"), (dict(rstd=None), "rstd is NULL"), (dict(d_weight=at(7) + 2), "misaligned"),
    (dict(d_x_stride=8), "stride"), (dict(d_y_stride=-1), "stride"), (dict(d_x=at(0) + 2), "overlaps"),
    (dict(d_weight=at(4)), "overlaps"), (dict(d_weight=at(8)), "overlaps"), (dict(d_bias=at(6)), "overlaps"),
    (dict(ws=at(3) + 16), "overlaps"), (dict(ws=at(7) + 16), "overlaps"), (dict(d_x=at(0), d_x_stride=32), "overlaps"),
])
def test_norm_grad_refusals(over, text):
    refused(norm_grad_call(**over), text)


def test_no_rows_without_sums_are_nothing_to_do():
    gone = dict(n=0, d_y=None, x=None, d_total=None, mean=None, rstd=None)
    assert norm_grad_call(**gone, ws=None, d_weight=None, d_bias=None) == 0
    assert norm_grad_call(**gone, accumulate=1) == 0
    assert norm_call(n=0, x=None, y=None, weight=None, bias=None, mean=None, rstd=None) == 0


def test_null_arguments():
    refused(layers.library().zero_norm(None, None), "NULL arguments")
    refused(layers.library().zero_norm_grad(None, None, 0, None), "NULL arguments")


class Elsewhere:
    """What a tensor of another device looks like to the binding."""

    is_cuda, device, shape, nbytes = True, "cuda:7", (4, 8), 1 << 20

    def __init__(self, dtype):
        self.dtype = dtype

    def get_device(self):
        return 7

    def stride(self):
        return (8, 1)

    def numel(self):
        return 32

    def is_contiguous(self):
        return True


def test_the_binding_takes_device_tensors_only():
    torch = pytest.importorskip("torch")
    x, t = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int64)
    for call in (lambda: layers.zero_embedding(t, x, x), lambda: layers.zero_token_order(t, 5, x),
                 lambda: layers.zero_embedding_grad(x, 5, x, x, x), lambda: layers.zero_norm(x, x),
                 lambda: layers.zero_norm_grad(x, x, x, x), lambda: layers.zero_norm([1.0], None)):
        with pytest.raises(TypeError, match="device memory expected"):
            call()
    far, ids = Elsewhere(torch.float32), Elsewhere(torch.int64)
    for call in (lambda: layers.zero_embedding(ids, far, far), lambda: layers.zero_token_order(ids, 5, far),
                 lambda: layers.zero_embedding_grad(far, 5, far, far, far), lambda: layers.zero_norm(far, far),
                 lambda: layers.zero_norm_grad(far, far, far, far)):
        with pytest.raises(ValueError, match="is on cuda:7, the current device is"):
            call()
