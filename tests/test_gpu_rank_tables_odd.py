"""An accumulated step with token tables of odd sizes: pieces and parts that begin
and end at any element. Whole numbers, so every sum is exact in any order."""

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from fsdp_sharded_mixed_zero_amd import synth  # noqa: E402
from fsdp_sharded_mixed_zero_amd.rank import RankShard  # noqa: E402
from layer_cases import DEV, generator  # noqa: E402

DIM, ROWS, MICRO = 37, 101, 3
SIZES = (19, ROWS * DIM, DIM, 641, 3 * DIM, 5001)
TABLES = {1: {"dim": DIM, "tokens": 50}, 4: {"dim": DIM, "tokens": 9, "dense": True}}


def whole(gen, *shape):
    return torch.randint(-8, 9, shape, generator=gen, device=DEV)


@pytest.mark.parametrize("n_d,rank", [(1, 0), (4, 0), (4, 1), (4, 2), (4, 3)])
@pytest.mark.parametrize("bucket", [0, 777])
def test_accumulator_of_odd_tables(n_d, rank, bucket):
    wl = synth.Workload("odd", SIZES, n_d=n_d, rank=rank, align=16, seed=3)
    rs = RankShard(wl, accum_steps=MICRO, tables=TABLES, bucket=bucket)
    want = torch.zeros(max(rs.info["padded"], sum(SIZES)), device=DEV)
    gen = generator(n_d * 10 + rank)

    def before_micro(mb):
        off, out = 0, {}
        for i, size in enumerate(SIZES):
            dense, t = whole(gen, size), TABLES.get(i)
            if rs.grads[i] is not None:
                rs.grads[i].copy_(dense)
            if t is None or t.get("dense"):
                want[off:off + size] += dense
            if t is not None and not (i == 1 and mb == 1):      # one micro-batch without tokens
                tokens = torch.randint(-1, size // DIM + 1, (t["tokens"] - mb,), generator=gen, device=DEV)
                d_out = whole(gen, len(tokens), DIM).to(torch.bfloat16)
                out[i] = (tokens, d_out)
                inside = (tokens >= 0) & (tokens < size // DIM)
                want[off:off + size].view(-1, DIM).index_add_(0, tokens[inside], d_out[inside].float())
            off += size
        return out

    rs.step(1, before_micro=before_micro)
    lo = rs.info["shard_begin"]
    assert torch.equal(rs.acc, want[lo:lo + rs.shard])
    assert int(rs.acc.count_nonzero()) > 0
