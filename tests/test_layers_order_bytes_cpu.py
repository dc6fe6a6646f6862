"""An order buffer made for fewer tokens than the gradient reads is refused by the
binding: the library is given its address only."""

import os

import pytest

torch = pytest.importorskip("torch")

from fsdp_sharded_mixed_zero_amd import layers, zero  # noqa: E402
from test_layers_integers_cpu import Null, device  # noqa: E402,F401

pytestmark = pytest.mark.skipif(not os.path.exists(zero.LIB_PATH),
                                reason="libzero_mi355x.so not built (run __graft_entry__.build())")


@pytest.mark.parametrize("made_for,n", [(0, 1), (8, 9), (4000, 4001), (12288, 12289), (20000, 24000)])
def test_an_order_for_fewer_tokens(made_for, n, device):  # noqa: F811
    order, ws = Null(torch.int32, 64), Null(torch.float32, 64)
    d_out, grad = Null(torch.float32, n, 8), Null(torch.float32, 40)
    assert layers.zero_token_order_bytes(made_for, 5) < layers.zero_token_order_bytes(n, 5)
    order.nbytes = layers.zero_token_order_bytes(made_for, 5)
    with pytest.raises(ValueError, match="order: .* bytes given, the call reaches"):
        layers.zero_embedding_grad(order, 5, d_out, grad, ws)
    order.nbytes = layers.zero_token_order_bytes(n, 5)
    with pytest.raises(zero.ZeroError, match="NULL order"):          # enough: the library's own checks
        layers.zero_embedding_grad(order, 5, d_out, grad, ws)
