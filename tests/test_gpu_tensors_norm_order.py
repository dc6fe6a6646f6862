"""The sum of squares of a list has the same bits wherever the gradients lie:
also where they are so far apart that one launch cannot carry their addresses,
and a launch then ends inside a block's four chunks of 4096 elements."""

import numpy as np
import pytest

from fsdp_sharded_mixed_zero_amd import tensors, zero
from oracle import step as O

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda"
LENS = [2 * 4096 + 7, 4096, 5, 3 * 4096, 1, 0, 9000, 4097, 20_000, 5 * 4096, 100, 3 * 4096 + 1, 4096]
APART = (1 << 32) + 64      # elements: beyond 32-bit steps between addresses an odd number of elements apart
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def patterns(n):
    """Which of n tensors lie far away."""
    yield "alternate", [i % 2 == 1 for i in range(n)]
    yield "second half", [i >= n // 2 for i in range(n)]
    for k in range(0, n, 3):
        yield f"only {k}", [i == k for i in range(n)]
    rng = np.random.default_rng(n)
    for k in range(4):
        yield f"random {k}", [bool(x) for x in rng.random(n) < 0.4]


@pytest.fixture(scope="module")
def arena():
    """Room for near tensors at odd elements and far ones at even elements, for both types."""
    x = torch.empty(4 * (APART + (1 << 23)), dtype=torch.uint8, device=DEV)
    yield x
    del x
    torch.cuda.empty_cache()


def place(arena, dtype, grads, far):
    flat = arena.view(dtype)
    at = {False: 1, True: APART}
    out = []
    for g, f in zip(grads, far):
        x = flat[at[f]:at[f] + g.numel()]
        x.copy_(g)
        at[f] += (g.numel() + 1) // 2 * 2 + 2
        out.append(x)
    return out


def norm(lst, grads):
    """The norm of a call, then accumulated once more; nothing outside the workspace is written."""
    need = tensors.zero_tensors_sqnorm_workspace_bytes(lst) // 8
    ws = torch.full((need + 2,), float("nan"), dtype=torch.float64, device=DEV)
    out = torch.zeros(2, dtype=torch.float64, device=DEV)
    ptrs = zero.pointer_array([g if g is not None and g.numel() else None for g in grads])
    tensors.zero_tensors_sqnorm(lst, ptrs, out[:1], False, ws[1:-1])
    tensors.zero_tensors_sqnorm(lst, ptrs, out[1:], False, ws[1:-1])
    tensors.zero_tensors_sqnorm(lst, ptrs, out[1:], True, ws[1:-1])
    once, twice = out.tolist()
    assert twice == once + once
    assert torch.isnan(ws[0]) and torch.isnan(ws[-1])
    return once


def make(lens, dtype, seed):
    rng = np.random.default_rng(seed)
    grads = [torch.from_numpy((rng.standard_normal(n) ** 3).astype(np.float32)).to(DEV).to(TYPES[dtype]) for n in lens]
    p, m, v = ([torch.zeros(n, device=DEV) for n in lens] for _ in range(3))
    return grads, tensors.zero_tensors(p, m, v, grad_dtype=TYPES[dtype])


@pytest.mark.parametrize("dtype", TYPES)
def test_few_tensors(arena, dtype):
    grads, lst = make(LENS, dtype, 1)
    want = norm(lst, place(arena, TYPES[dtype], grads, [False] * len(LENS)))
    exact = sum(O.sqnorm_f32(g.float().cpu().numpy()) for g in grads)
    assert abs(want - exact) <= sum(LENS) * 2.0 ** -53 * exact     # each of the additions rounds by 2^-53 at most
    differ = [name for name, far in patterns(len(LENS))
              if norm(lst, place(arena, TYPES[dtype], grads, far)) != want]
    assert not differ


@pytest.mark.parametrize("dtype", TYPES)
def test_more_tensors_than_a_launch(arena, dtype):
    """Cuts by the addresses beside those after 768 tensors."""
    lens = [int(n) for n in np.random.default_rng(5).integers(0, 9000, 1700)]
    grads, lst = make(lens, dtype, 2)
    want = norm(lst, place(arena, TYPES[dtype], grads, [False] * len(lens)))
    rng = np.random.default_rng(6)
    for share in (0.5, 0.01):
        far = [bool(x) for x in rng.random(len(lens)) < share]
        assert norm(lst, place(arena, TYPES[dtype], grads, far)) == want


def test_missing_gradients_far_apart(arena):
    """A missing gradient adds nothing, far away or near."""
    grads, lst = make(LENS, "bf16", 3)
    gone = lambda views: [None if i in (1, 6) else g for i, g in enumerate(views)]  # noqa: E731
    want = norm(lst, gone(place(arena, torch.bfloat16, grads, [False] * len(LENS))))
    for _, far in patterns(len(LENS)):
        assert norm(lst, gone(place(arena, torch.bfloat16, grads, far))) == want


def test_far_apart_from_a_graph(arena):
    """Replays, whatever the workspace holds before each, between eager norms of the same gradients near each other."""
    far = [i % 2 == 1 for i in range(len(LENS))]
    grads, lst = make(LENS, "bf16", 7)
    ws = torch.empty(tensors.zero_tensors_sqnorm_workspace_bytes(lst) // 8, dtype=torch.float64, device=DEV)
    out = torch.zeros(1, dtype=torch.float64, device=DEV)
    views = place(arena, torch.bfloat16, grads, far)
    ptrs = zero.pointer_array([g if g.numel() else None for g in views])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tensors.zero_tensors_sqnorm(lst, ptrs, out, False, ws)
    for k in range(4):
        for x, g in zip(views, grads):
            g.mul_(-0.5 - k)
            x.copy_(g)
        ws.fill_(float("nan") if k % 2 else 1e30)
        graph.replay()
        torch.cuda.synchronize()
        got = out.item()
        near = [g.clone() for g in grads]
        assert norm(lst, near) == got
