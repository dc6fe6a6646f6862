"""The table gradients of an accumulated step, on the host: which stream the
allocator is told of for the tensors of a micro-batch. The calls are stand-ins
that note what they are given; nothing is launched."""

import pytest

torch = pytest.importorskip("torch")

from fsdp_sharded_mixed_zero_amd import rank as R  # noqa: E402

DIM, ROWS = 4, 6


class Stream:
    cuda_stream = 77


class Given:
    """A tensor as the step sees one."""

    def __init__(self, what, log, *shape):
        self.what, self.log, self.shape = what, log, shape

    def numel(self):
        return self.shape[0]

    def record_stream(self, stream):
        self.log.append((self.what, stream))


def shard(log, monkeypatch):
    monkeypatch.setattr(R.layers, "zero_token_order",
                        lambda tokens, rows, order, stream=None: log.append(("sort", stream)))
    monkeypatch.setattr(R.layers, "zero_embedding_grad", lambda *a, stream=None, **k: log.append(("gradient", stream)))
    rs = R.RankShard.__new__(R.RankShard)
    rs.device = torch.device("cuda")
    rs.acc = torch.zeros(ROWS * DIM)
    rs.segments = [(0, 0, 0, ROWS * DIM)]
    rs.tables = {0: {"dim": DIM, "rows": ROWS, "tokens": 8, "dense": False, "order": None, "workspace": None,
                     "none": (Given("none", [], 0), Given("none", [], 0, DIM))}}
    return rs


@pytest.mark.parametrize("kind", ["stream", "handle", "current"])
def test_the_allocator_is_told_of_the_stream_that_reads_a_micro_batch(kind, monkeypatch):
    """Each tensor right behind the call that reads it, so also where a later call refuses its own."""
    log, there = [], Stream()
    monkeypatch.setattr(R.torch.cuda, "ExternalStream", lambda handle, device=None: ("external", handle, device))
    monkeypatch.setattr(R.torch.cuda, "current_stream", lambda *a: "current")
    rs = shard(log, monkeypatch)
    given, seen = {"stream": (there, there), "handle": (77, ("external", 77, rs.device)), "current": (None, "current")}[kind]
    rs._accumulate_tables({0: (Given("tokens", log, 5), Given("d_out", log, 5, DIM))}, True, given)
    assert log == [("sort", given), ("tokens", seen), ("gradient", given), ("d_out", seen)]


def test_tokens_are_held_where_the_gradient_is_refused(monkeypatch):
    log, there = [], Stream()
    rs = shard(log, monkeypatch)

    def refuse(*a, **k):
        raise TypeError("d_out")

    monkeypatch.setattr(R.layers, "zero_embedding_grad", refuse)
    with pytest.raises(TypeError):
        rs._accumulate_tables({0: (Given("tokens", log, 5), Given("d_out", log, 5, DIM))}, True, there)
    assert log == [("sort", there), ("tokens", there)]
