"""A list's table: written on a stream of the caller's while another stream
still writes memory that it has freed."""

import pytest

from fsdp_sharded_mixed_zero_amd import tensors, zero

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda"


def make(columns, stream=None):
    return tensors.zero_tensors(*columns, stream=stream)


@pytest.mark.parametrize("by_handle", [False, True])
def test_a_list_made_on_another_stream_beside_pending_work(by_handle):
    columns = [[torch.ones(n, device=DEV) for n in (700, 5, 3000)] for _ in range(3)]
    size = make(columns).table.numel()      # a list dropped at once
    side = torch.cuda.Stream()
    busy = torch.randn(4096, 4096, device=DEV)
    torch.cuda.synchronize()
    for _ in range(20):
        busy = busy @ busy * 1e-3
    freed = [torch.full((size,), -1, dtype=torch.int64, device=DEV) for _ in range(8)]   # written after the products
    del freed
    lst = make(columns, side.cuda_stream if by_handle else side)
    torch.cuda.synchronize()
    want = make(columns)
    # compared before anything reads it: the records name the same tensors
    assert torch.equal(lst.table.view(torch.uint8)[:tensors.zero_tensors_table_bytes(lst)],
                       want.table.view(torch.uint8)[:tensors.zero_tensors_table_bytes(want)])
    sums = torch.full((1,), 0.25, dtype=torch.float64, device=DEV)
    grads = [torch.full_like(p, 0.5) for p in columns[0]]
    torch.cuda.synchronize()
    tensors.zero_tensors_adamw_step(lst, grads, zero.hparams(lr=0.25, step=1), sums, 1, stream=side)
    torch.cuda.synchronize()
    assert all(bool((p < 1).all()) for p in columns[0])
