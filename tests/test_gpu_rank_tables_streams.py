"""An accumulated step with a token table on a stream that is not the one its
micro-batches are made on."""

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from fsdp_sharded_mixed_zero_amd import synth  # noqa: E402
from fsdp_sharded_mixed_zero_amd.rank import RankShard  # noqa: E402
from layer_cases import DEV, draw_tokens, generator, normal  # noqa: E402

DIM, ROWS, TOKENS, MICRO = 264, 3001, 20000, 4
SIZES = (ROWS * DIM, DIM, 30 * DIM)


@pytest.mark.parametrize("kind", ["stream", "handle"])
def test_micro_batches_may_be_dropped_at_once(kind):
    """Each micro-batch's tensors are temporaries of the current stream, dropped when the next one is made, which
    allocates as many bytes and overwrites them: the accumulator is that of a step on the current stream."""
    wl = synth.Workload("streams", SIZES, n_d=1, rank=0, align=16, grad_std=1e-2, seed=3)
    tables = {0: {"dim": DIM, "tokens": TOKENS}}
    kept = [(draw_tokens(TOKENS, ROWS, mb), normal(generator(mb), TOKENS, DIM, dtype=torch.bfloat16)) for mb in range(MICRO)]
    here, there = RankShard(wl, accum_steps=MICRO, tables=tables), RankShard(wl, accum_steps=MICRO, tables=tables)
    here.step(1, before_micro=lambda mb: {0: kept[mb]})
    side = torch.cuda.Stream()
    torch.cuda.synchronize()

    def before_micro(mb):
        junk = [torch.full_like(t, 0) for t in kept[mb]]      # in the memory that is free by now
        del junk
        tokens, d_out = (t.clone() for t in kept[mb])
        side.wait_stream(torch.cuda.current_stream())
        return {0: (tokens, d_out)}

    there.step(1, stream=side if kind == "stream" else side.cuda_stream, before_micro=before_micro)
    junk = [torch.full_like(t, 0) for t in kept[0]]
    torch.cuda.synchronize()
    assert torch.equal(here.acc, there.acc) and torch.equal(here.param_shard, there.param_shard)
    assert all(int(t.count_nonzero()) == 0 for t in junk)


def test_a_step_on_the_default_streams_handle():
    wl = synth.Workload("streams", SIZES, n_d=1, rank=0, align=16, grad_std=1e-2, seed=3)
    tables = {0: {"dim": DIM, "tokens": 50}}
    given = (draw_tokens(50, ROWS, 1), normal(generator(1), 50, DIM, dtype=torch.bfloat16))
    a, b = RankShard(wl, accum_steps=2, tables=tables), RankShard(wl, accum_steps=2, tables=tables)
    a.step(1, before_micro=lambda mb: {0: given})
    b.step(1, stream=torch.cuda.default_stream().cuda_stream, before_micro=lambda mb: {0: tuple(t.clone() for t in given)})
    torch.cuda.synchronize()
    assert torch.equal(a.acc, b.acc) and torch.equal(a.param_shard, b.param_shard)
