"""A rank whose shard holds padding only, its slice held tensor by tensor."""

import pytest

from fsdp_sharded_mixed_zero_amd import synth, zero
from fsdp_sharded_mixed_zero_amd.rank import TensorRank

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [32, 8])
def test_a_rank_of_padding_only(bits):
    """As RankShard has it: its sum of squares is 0 and its step changes nothing."""
    wl = synth.Workload("short", (100,), n_d=4, rank=3, m_std=1e-4, v_std=1e-8, step=7)
    assert not zero.zero_layout(wl.sizes, wl.n_d, wl.rank, wl.align).segments
    r = TensorRank(wl, state_bits=bits)
    assert r.list.state_bits == bits
    others = r.rank_sq.clone()
    assert float(others.sum()) > 0
    r.rank_sq[r.rank] = 5.0
    r.step(wl.step)
    torch.cuda.synchronize()
    assert torch.equal(r.rank_sq, others)
    assert r.bytes_per_step() == {"sqnorm": 0, "adamw": 0}
