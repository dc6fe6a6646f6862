"""Group indices out of range: the library's to refuse, and the binding's where
the record's 32 bits would hold another one."""

import pytest

from fsdp_sharded_mixed_zero_amd import tensors, zero

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("group", [8, -1, 1 << 32, (1 << 32) + 3, -(1 << 32)])
def test_groups_out_of_range(group):
    cols = [[torch.zeros(8, device="cuda") for _ in range(2)] for _ in range(3)]
    with pytest.raises((ValueError, zero.ZeroError), match="group"):
        tensors.zero_tensors(*cols, group=[0, group])
    assert tensors.zero_tensors(*cols, group=[7, 0]).n_tensors == 2
