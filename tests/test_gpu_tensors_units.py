"""The three ways the 8-bit kernels share out a list, by its number of units
(1024 elements of one tensor) and of partial ones: four, two or one wave a
unit. Each list against the fp64 definition: step, import and export."""

import numpy as np
import pytest

from fsdp_sharded_mixed_zero_amd import tensors, zero
from oracle import state8 as S8
from tensor_lists import Arena, Case
from test_gpu_tensors import check8, check_codes, run_step

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def ragged(n, low, high, seed):
    """n lengths of every kind of end: whole units, whole blocks, inside a block."""
    rng = np.random.default_rng(seed)
    out = rng.integers(low, high, n)
    out[::5] = out[::5] // 1024 * 1024
    out[1::5] = out[1::5] // 256 * 256
    return [int(x) for x in out]


LISTS = {
    "four waves, 1024 units": [1024 * 1000, 1, 255, 256, 257, 511, 769, 1023] + [700] * 17,
    "two waves, 1025 units": [1024 * 1000, 1, 255, 256, 257, 511, 769, 1023] + [700] * 18,
    "two waves, ragged": ragged(250, 1, 12000, 1),
    "two waves, many partial units": ragged(700, 2000, 9000, 2),
    "one wave, few partial units": [1024 * 1500 + 700, 5, 1024 * 400 + 257, 300],
}


def units(lens):
    return sum(-(-n // 1024) for n in lens)


def test_the_lists_are_what_they_are_called():
    n = {k: units(v) for k, v in LISTS.items()}
    assert n["four waves, 1024 units"] == 1024 and n["two waves, 1025 units"] == 1025
    assert 1024 < n["two waves, ragged"] <= 1792 < n["two waves, many partial units"]
    many = LISTS["two waves, many partial units"]
    assert n["two waves, many partial units"] <= 20 * sum(x % 1024 != 0 for x in many) and len(many) <= 768
    one = LISTS["one wave, few partial units"]
    assert n["one wave, few partial units"] > max(1792, 20 * sum(x % 1024 != 0 for x in one))


@pytest.mark.parametrize("name", LISTS)
@pytest.mark.parametrize("grad,param", [("bf16", "bf16"), ("f32", "f32")])
def test_step8(name, grad, param):
    case = Case(LISTS[name], 8, param, grad, seed=41, missing=(3,), groups=2).to_device()
    check8(case, *run_step(case, groups=2)[:3])


@pytest.mark.parametrize("name", LISTS)
def test_import_and_export(name):
    lens = LISTS[name]
    case = Case(lens, 8, seed=42).to_device()
    m, v = Arena(case.m, "f32"), Arena(case.v, "f32")
    tensors.zero_tensors_state_import(case.list, m.views, v.views)
    torch.cuda.synchronize()
    got = {k: case.A[k].tensors() for k in ("m", "m_scale", "v", "v_scale")}
    case.check_guards()
    out = [Arena([np.zeros(n, np.float32) for n in lens], "f32") for _ in range(2)]
    tensors.zero_tensors_state_export(case.list, zero.pointer_array([t if n else None for t, n in
                                                                     zip(out[0].views, lens)]), out[1].views)
    torch.cuda.synchronize()
    back = [a.tensors() for a in out]
    for a in out:
        a.check_guards("export")
    for i in range(len(lens)):
        now = [got[k][i] for k in ("m", "m_scale", "v", "v_scale")]
        check_codes(now, S8.encode(case.m[i].astype(np.float64), case.v[i].astype(np.float64)), f"tensor {i}")
        m64, v64 = S8.decode(*now)
        assert np.array_equal(back[0][i], m64.astype(np.float32)), f"m {i}"
        assert np.array_equal(back[1][i], v64.astype(np.float32)), f"v {i}"
