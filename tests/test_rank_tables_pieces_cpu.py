"""The dense pieces of an accumulated step with token tables of odd sizes, on the
host: they cover all but the tables, and all but a few elements of each are added from
an aligned element on, where the call takes vectors."""

import os

import pytest

torch = pytest.importorskip("torch")

from fsdp_sharded_mixed_zero_amd import rank as R  # noqa: E402
from fsdp_sharded_mixed_zero_amd import synth, zero  # noqa: E402

pytestmark = pytest.mark.skipif(not os.path.exists(zero.LIB_PATH),
                                reason="libzero_mi355x.so not built (run __graft_entry__.build())")

DIM = 37
SIZES = (19, 101 * DIM, DIM, 641, 3 * DIM, 5001)
TABLES = {1: {"dim": DIM, "tokens": 4}, 4: {"dim": DIM, "tokens": 4}}


@pytest.mark.parametrize("n_d,rank", [(1, 0), (4, 0), (4, 1), (4, 3)])
@pytest.mark.parametrize("bucket", [0, 1024, 777])
def test_pieces_are_added_from_aligned_elements_on(n_d, rank, bucket, monkeypatch):
    monkeypatch.setattr(R.zero, "pointer_array", lambda tensors: None)
    wl = synth.Workload("odd", SIZES, n_d=n_d, rank=rank, align=16)
    rs = R.RankShard(wl, device="cpu", fill=False, accum_steps=2, tables=TABLES, bucket=bucket)
    packed, added = [], []
    monkeypatch.setattr(R.zero, "zero_pack_grads", lambda lay, ptrs, shard, b, n, stream: packed.append((b, n)))

    def accumulate(grad, acc, n, first, stream):
        at = (acc.data_ptr() - rs.acc.data_ptr()) // 4
        assert at == (grad.data_ptr() - rs.grad_shard.data_ptr()) // 2
        added.append((at, n))

    monkeypatch.setattr(R.zero, "zero_accumulate_grads", accumulate)
    for name in ("zero_shard_sqnorm_f32", "zero_adamw_step_f32grad_unpack"):
        monkeypatch.setattr(R.zero, name, lambda *a, **k: None)
    monkeypatch.setattr(rs, "_accumulate_tables", lambda *a: None)
    rs._step_accumulated(None, rs.rank_sq[:1], rs.pieces(), None, lambda phase, fn: fn(), None)
    tables = torch.zeros(rs.shard, dtype=torch.int32)
    for i, _, d, n in rs.segments:
        if i in TABLES:
            tables[d:d + n] = 2
    for calls in (packed, added):
        times = tables.clone()
        for b, n in calls:
            times[b:b + n] += 1
        assert (times == 2).all()          # each other element once a micro-batch
    assert all(b % 8 == 0 or n < 8 for b, n in added)
    if n_d == 1:
        assert any(b % 8 for b, n in packed)
