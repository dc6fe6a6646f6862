"""TensorRank's state arrays rebound between steps, as a restored checkpoint does."""

import pytest

from fsdp_sharded_mixed_zero_amd import synth
from fsdp_sharded_mixed_zero_amd.rank import TensorRank

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ODD = synth.Workload("odd", tuple([5000, 33, 1, 70001, 257, 4096, 12345, 999]), n_d=3, rank=1, m_std=1e-4, v_std=1e-8,
                     step=7)
NAMES = {32: ("master", "m", "v"), 8: ("master", "m8", "v8", "m_scale", "v_scale")}


@pytest.mark.parametrize("bits", [32, 8])
def test_rebound_arrays_are_the_ones_a_step_updates(bits):
    """A restored checkpoint: other arrays under the same names."""
    a, b = TensorRank(ODD, state_bits=bits), TensorRank(ODD, state_bits=bits)
    a.step(ODD.step)
    b.step(ODD.step)
    old = {}
    for k in NAMES[bits]:
        old[k] = getattr(b, k)
        setattr(b, k, old[k].clone())
    kept = {k: x.clone() for k, x in old.items()}
    for t in (ODD.step + 1, ODD.step + 2):
        a.step(t)
        b.step(t)
    torch.cuda.synchronize()
    for k in NAMES[bits]:
        assert torch.equal(getattr(a, k).view(torch.uint8), getattr(b, k).view(torch.uint8)), k
        assert torch.equal(old[k].view(torch.uint8), kept[k].view(torch.uint8)), f"{k}: the old array was written"
    for i in a.touched:
        assert torch.equal(a.params[i].view(torch.int16), b.params[i].view(torch.int16))


def test_arrays_that_do_not_fit_are_refused():
    b = TensorRank(ODD, fill=False)
    b.m = b.m[:-1].clone()
    with pytest.raises(ValueError, match="m "):
        b.step(ODD.step)
    b = TensorRank(ODD, fill=False)
    b.v = b.v.double()
    with pytest.raises(TypeError, match="v "):
        b.step(ODD.step)


def test_rebound_arrays_are_refused_while_capturing():
    """The list's new table would be written by the graph's replays only."""
    b = TensorRank(ODD)
    b.step(ODD.step)
    b.m = b.m.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with pytest.raises(RuntimeError, match="rebound"):
        with torch.cuda.graph(g):
            b.step(ODD.step)
    torch.cuda.synchronize()
    b.step(ODD.step)
    torch.cuda.synchronize()


@pytest.mark.parametrize("bits", [32, 8])
def test_a_graph_captured_before_goes_on_with_its_arrays(bits):
    """Its list's table is still there after the rank's list was made again and memory given out."""
    a, b = TensorRank(ODD, state_bits=bits), TensorRank(ODD, state_bits=bits)
    a.step(ODD.step)
    b.step(ODD.step)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.step(ODD.step)
    old = {k: getattr(b, k) for k in NAMES[bits]}
    size = b.list.table.numel()
    for k in NAMES[bits]:
        setattr(b, k, old[k].clone())
    b.step(ODD.step)
    filled = [torch.full((size,), -1, dtype=torch.int64, device="cuda") for _ in range(8)]
    for _ in range(3):
        a.step(ODD.step)
        graph.replay()
        torch.cuda.synchronize()
        for k in NAMES[bits]:
            assert torch.equal(getattr(a, k).view(torch.uint8), old[k].view(torch.uint8)), k
    assert all(int(f.min()) == -1 for f in filled)
