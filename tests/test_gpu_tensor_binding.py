"""The tensor-list binding where a list's arguments are unusual: tensors
without elements that have no state, a table that the caller keeps by its
address, another table for the same list."""

import numpy as np
import pytest

from fsdp_sharded_mixed_zero_amd import tensors, zero
from tensor_lists import Case
from test_gpu_tensors import check8, check32, run_step

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [32, 8])
def test_empty_tensors_without_state(bits):
    """A first tensor of no elements may have None for its moments."""
    case = Case([0, 700, 0, 5], bits, seed=31).to_device()
    views = lambda k: [t if n else None for t, n in zip(case.A[k].views, case.lens)] if k in case.A else None  # noqa: E731
    case.list = tensors.zero_tensors(case.A["param"].views, views("m"), views("v"), master=views("master"),
                                     m_scale=views("m_scale"), v_scale=views("v_scale"))
    assert case.list.state_bits == bits
    hps, steps, coef, parts = run_step(case)
    check8(case, hps, steps, coef) if bits == 8 else check32(case, hps, steps, coef, parts, 4)


def test_a_list_of_empty_tensors_without_state():
    p = [torch.empty(0, dtype=torch.float32, device="cuda") for _ in range(2)]
    lst = tensors.zero_tensors(p, [None, None], [None, None])
    out = torch.full((1,), 7.0, dtype=torch.float64, device="cuda")
    ws = torch.empty(1, dtype=torch.float64, device="cuda")
    tensors.zero_tensors_sqnorm(lst, p, out, False, ws)
    assert float(out) == 0.0


@pytest.mark.parametrize("by_address", [False, True])
def test_another_table(by_address):
    """A list bound to a second table, a tensor's or an address's, steps as with its own."""
    case = Case([700, 1, 4000], 32, seed=32).to_device()
    nbytes = tensors.zero_tensors_table_bytes(case.list)
    table = torch.zeros(-(-nbytes // 8), dtype=torch.int64, device="cuda")
    tensors.zero_tensors_upload(case.list, table.data_ptr() if by_address else table, nbytes)
    hps, steps, coef, parts = run_step(case)
    check32(case, hps, steps, coef, parts, 4)


def test_sizes_beyond_the_tensors_are_refused():
    case = Case([9000], 32, seed=33).to_device()
    small = torch.zeros(1, dtype=torch.float64, device="cuda")
    need = tensors.zero_tensors_sqnorm_workspace_bytes(case.list)
    with pytest.raises(ValueError, match="workspace"):
        tensors.zero_tensors_sqnorm(case.list, case.grad_ptrs, small, False, small, ws_bytes=need)
    with pytest.raises(ValueError, match="table"):
        tensors.zero_tensors_upload(case.list, small, tensors.zero_tensors_table_bytes(case.list))
    with pytest.raises(zero.ZeroError):
        tensors.zero_tensors_sqnorm(case.list, case.grad_ptrs, small, False, small)
    assert np.array_equal(case.A["m"].bits(), case.A["m"].before)
