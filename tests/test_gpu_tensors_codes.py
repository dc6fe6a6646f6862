"""Every scale and every byte of the 8-bit state that the kernels write, in
blocks whose scale is a neighbour of the definition's too (state8_codes)."""

import numpy as np
import pytest

import state8_codes
from fsdp_sharded_mixed_zero_amd import tensors
from oracle import state8 as S8
from tensor_lists import Arena, Case
from test_gpu_tensors import RAGGED, many_lens, run_step
from test_gpu_tensors_small_roots import spread
from test_gpu_tensors_units import LISTS

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def check_step(case, hps, steps, coef):
    got = {k: case.A[k].tensors() for k in ("m", "m_scale", "v", "v_scale")}
    other = 0
    for i, n in enumerate(case.lens):
        if i in case.missing or n == 0:
            continue
        hp, step = hps[case.group[i]], steps[case.group[i]]
        _, m1, v1, _ = S8.adamw8_step(case.grads[i], case.master[i], *case.state[i], step, hp, coef)
        other += state8_codes.check([got[k][i] for k in ("m", "m_scale", "v", "v_scale")], m1, v1,
                                    state8_codes.step_slack(case.grads[i], *case.state[i], hp, coef), f"tensor {i}")
    # a maximum lies within 2^-48 of itself of a border in one block of 2^24
    assert other <= 2


def check_import(case, ms, vs):
    got = {k: case.A[k].tensors() for k in ("m", "m_scale", "v", "v_scale")}
    for i in range(len(case.lens)):
        assert state8_codes.check([got[k][i] for k in ("m", "m_scale", "v", "v_scale")], ms[i], vs[i],
                                  None, f"tensor {i}") == 0


@pytest.mark.parametrize("grad,param", [("bf16", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("align", [1, 64])
def test_step_ragged(grad, param, align):
    case = Case(RAGGED, 8, param, grad, seed=align, missing=(4, 19), groups=3, align=align).to_device()
    check_step(case, *run_step(case, groups=3)[:3])


def test_step_of_900_tensors():
    case = Case(many_lens(), 8, seed=2, missing=range(0, 900, 11), groups=8).to_device()
    check_step(case, *run_step(case, groups=8, n_ranks=70)[:3])


@pytest.mark.parametrize("name", LISTS)
def test_step_by_units(name):
    case = Case(LISTS[name], 8, seed=43, missing=(3,), groups=2).to_device()
    check_step(case, *run_step(case, groups=2)[:3])


@pytest.mark.parametrize("scale", [1e-30, 3e-23, 1e-18, 1e-9, 1e6, 1e15])
def test_step_magnitudes(scale):
    case = Case([700, 256], 8, grad="f32", seed=7, m_std=scale, v_std=scale ** 2, g_std=scale).to_device()
    check_step(case, *run_step(case, max_norm=0.0)[:3])


@pytest.mark.parametrize("lo,hi", [(-120, 0), (-149, -100), (-80, 40), (0, 60)])
def test_step_over_many_binades(lo, hi):
    case = Case([1024, 1, 1500, 255], 8, grad="f32")
    case.grads = case.grad_bits = [spread(n, lo, hi, i) for i, n in enumerate(case.lens)]
    case.state = [tuple(np.zeros_like(x) for x in s) for s in case.state]
    case.to_device()
    check_step(case, *run_step(case, step=1, max_norm=0.0, eps=0.0)[:3])


def test_step_of_zero_gradients_and_moments():
    """Rows without a token: whole blocks, single elements, and moments that stay zero beside ones that do not."""
    lens = [4096, 700, 1024 * 1200, 5]
    case = Case(lens, 8, grad="f32", seed=19)
    rng = np.random.default_rng(20)
    for i, n in enumerate(lens):
        off = rng.random(n) < 0.5
        off[:n // 3] = True
        case.grads[i][off] = 0.0
        m, v = case.m[i].copy(), case.v[i].copy()
        m[off & (np.arange(n) % 3 == 0)] = 0.0
        v[off] = 0.0
        case.state[i] = S8.encode(m, v)
    case.grad_bits = case.grads
    case.to_device()
    check_step(case, *run_step(case)[:3])
    v = case.A["v"].tensors()
    for i, g in enumerate(case.grads):
        assert ((v[i] > 0) == ((case.state[i][2] > 0) | (g != 0))).all()


@pytest.mark.parametrize("lens", [RAGGED, many_lens(), LISTS["one wave, few partial units"]], ids=["ragged", "900", "long"])
def test_import(lens):
    case = Case(lens, 8, seed=12).to_device()
    rng = np.random.default_rng(13)
    ms = [(rng.standard_normal(n) * 1e-3).astype(np.float32) for n in lens]
    vs = [(rng.random(n) ** 6 * 1e-6).astype(np.float32) for n in lens]
    m, v = Arena(ms, "f32"), Arena(vs, "f32")
    tensors.zero_tensors_state_import(case.list, m.views, v.views)
    torch.cuda.synchronize()
    check_import(case, ms, vs)
