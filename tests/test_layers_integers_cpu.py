"""Integers of the token-table and norm binding that do not fit the library's 64
bits are refused, not cut: 2^64 + 5 rows are not 5, and a first element of 2^64 is
not the table's first. The arrays are NULL, which the library refuses behind that."""

import os

import pytest

torch = pytest.importorskip("torch")

from fsdp_sharded_mixed_zero_amd import layers, zero  # noqa: E402

pytestmark = pytest.mark.skipif(not os.path.exists(zero.LIB_PATH),
                                reason="libzero_mi355x.so not built (run __graft_entry__.build())")

CUT = [2 ** 64 + 5, 2 ** 64, 2 ** 63, -2 ** 63 - 1, -2 ** 64 + 5]


class Null:
    """A tensor of device 0 without memory, as the binding sees one."""

    is_cuda, device, nbytes = True, "cuda:0", 1 << 20

    def __init__(self, dtype, *shape):
        self.dtype, self.shape = dtype, torch.Size(shape)

    def get_device(self):
        return 0

    def stride(self):
        return (self.shape[-1], 1)

    def numel(self):
        return self.shape.numel()

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0


@pytest.fixture
def device(monkeypatch):
    layers._load()
    monkeypatch.setattr(layers, "_device", lambda: 0)
    monkeypatch.setattr(layers, "_stream", lambda stream, dev: 0)


@pytest.mark.parametrize("k", CUT)
def test_sizes_of_buffers(k):
    for name in ("zero_token_order_bytes", "zero_embedding_grad_workspace_bytes", "zero_norm_grad_workspace_bytes"):
        for sizes in ((k, 50), (50, k)):
            with pytest.raises(ValueError, match="limits"):
                getattr(layers, name)(*sizes)


@pytest.mark.parametrize("k", CUT)
def test_rows_and_first_element(k, device):
    tokens, order, ws = Null(torch.int32, 5), Null(torch.int32, 64), Null(torch.float32, 64)
    d_out, grad = Null(torch.float32, 5, 8), Null(torch.float32, 40)
    with pytest.raises(ValueError, match="rows"):
        layers.zero_token_order(tokens, k, order)
    with pytest.raises(ValueError, match="rows"):
        layers.zero_embedding_grad(order, k, d_out, grad, ws)
    with pytest.raises(ValueError, match="first"):
        layers.zero_embedding_grad(order, 5, d_out, grad, ws, first=k)


@pytest.mark.parametrize("rows,first", [(2 ** 63 - 1, 0), (-2 ** 63, 0), (5, 2 ** 63 - 1), (5, -2 ** 63)])
def test_the_library_refuses_those_that_fit(rows, first, device):
    tokens, order, ws = Null(torch.int32, 5), Null(torch.int32, 64), Null(torch.float32, 64)
    d_out, grad = Null(torch.float32, 5, 8), Null(torch.float32, 40)
    with pytest.raises(zero.ZeroError, match="rows|first|elements"):
        layers.zero_embedding_grad(order, rows, d_out, grad, ws, first=first)
    if rows != 5:
        with pytest.raises(zero.ZeroError, match="rows"):
            layers.zero_token_order(tokens, rows, order)
