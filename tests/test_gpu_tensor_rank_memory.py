"""TensorRank's 8-bit moments while a rank is made: drawn and imported piece by
piece, as each tensor whole, without the shard's moments in fp32."""

import numpy as np
import pytest

from fsdp_sharded_mixed_zero_amd import synth, tensors
from fsdp_sharded_mixed_zero_amd.rank import RankShard, TensorRank
from oracle import state8 as S8

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda"
ODD = synth.Workload("odd", tuple([5000, 33, 1, 70001, 257, 4096, 12345, 999]), n_d=3, rank=1, m_std=1e-4, v_std=1e-8,
                     step=7)
BIG = synth.Workload("big", tuple([20_000_000, 1001, 9_000_003]), n_d=2, rank=0, m_std=1e-4, v_std=1e-8, step=7)


def allocated_while(make):
    """What make() returns, and the bytes that it had allocated at most."""
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    before = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    r = make()
    torch.cuda.synchronize()
    return r, torch.cuda.max_memory_allocated() - before


@pytest.mark.parametrize("fill", [False, True])
def test_an_8_bit_rank_never_holds_fp32_moments_of_the_shard(fill, monkeypatch):
    """Gradients, parameters, masters and the 8-bit state; to draw them, two
    pieces of the shard in fp32 and what drawing a piece takes beside it."""
    piece = 1 << 17
    monkeypatch.setattr(RankShard, "STATE_CHUNK", piece)
    if fill:      # the gradients of the other rank's slice are drawn in a buffer of the longest tensor
        monkeypatch.setattr(TensorRank, "fill_other_ranks", lambda self, step=None: None)
        monkeypatch.setattr(TensorRank, "fill_grads", lambda self, step: None)
    r, peak = allocated_while(lambda: TensorRank(BIG, state_bits=8, fill=fill))
    held = sum(2 * 2 * BIG.sizes[i] for i in r.touched) + (4 + 1 + 1) * r.shard + 8 * r.blocks
    assert peak <= held + 16 * 4 * piece + (4 << 20), (peak, held)       # the shard's fp32 moments would be 116 MB


@pytest.mark.parametrize("piece", [8192, 1 << 26])
@pytest.mark.parametrize("wl", [ODD, synth.WORKLOADS["tiny"]], ids=lambda w: w.name)
def test_the_8_bit_state_is_that_of_the_drawn_moments(wl, piece, monkeypatch):
    """Drawn in pieces that cut tensors and blocks, the moments come out as if each tensor were imported whole."""
    monkeypatch.setattr(RankShard, "STATE_CHUNK", piece)
    a, b = RankShard(wl, state_arrays=True), TensorRank(wl, state_bits=8)
    n = a.real
    assert torch.equal(a.master[:n].view(torch.int32), b.master[:n].view(torch.int32))
    m8, v8 = (x.view(torch.uint8).cpu().numpy() for x in (b.m8, b.v8))
    ms, vs = b.m_scale.cpu().numpy(), b.v_scale.cpu().numpy()
    m, v = (x.cpu().numpy().astype(np.float64) for x in (a.m, a.v))
    k = 0
    for _, _, d, n in b.segments:
        blocks = tensors.state8_blocks(n)
        got = m8[d:d + n], ms[k:k + blocks], v8[d:d + n], vs[k:k + blocks]
        for x, y in zip(got, S8.encode(m[d:d + n], v[d:d + n])):      # the maxima are exact: so are the scales
            assert np.array_equal(x, y)
        k += blocks


def test_fill_state_after_an_8_bit_rank_was_made_without():
    a, b = TensorRank(ODD, state_bits=8), TensorRank(ODD, state_bits=8, fill=False)
    b.fill_state()
    for k in ("master", "m8", "v8", "m_scale", "v_scale"):
        x, y = getattr(a, k), getattr(b, k)
        if k == "master":
            x, y = x[:a.real], y[:a.real]
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8)), k
