"""The 8-bit step where fp32 cannot resolve a second moment's root: eps = 0 or
nearly so, and roots of very different size in one block. Checked against the
float64 oracle, at the bounds of the ordinary elements."""

import numpy as np
import pytest

from oracle import state8 as S8
from tensor_lists import Case
from test_gpu_tensors import check8, run_step

pytestmark = pytest.mark.gpu


def spread(n, lo, hi, seed):
    """n non-zero values of both signs, evenly over the binades [lo, hi)."""
    rng = np.random.default_rng(seed)
    return (rng.choice([-1.0, 1.0], n) * 2.0 ** rng.uniform(lo, hi, n)).astype(np.float32)


def fresh(lens, lo, hi, **kw):
    """A list with zeroed moments, so that a first step's roots are as far apart as its gradients."""
    case = Case(lens, 8, grad="f32", **kw)
    case.grads = case.grad_bits = [spread(n, lo, hi, i) for i, n in enumerate(lens)]
    case.state = [tuple(np.zeros_like(x) for x in s) for s in case.state]
    return case.to_device()


@pytest.mark.parametrize("eps", [0.0, 1e-30, 1e-20, 1e-8])
@pytest.mark.parametrize("lo,hi", [(-120, 0), (-149, -100), (-80, 40), (0, 60)])
@pytest.mark.parametrize("param", ["bf16", "f32"])
def test_first_step_over_many_binades(lo, hi, eps, param):
    case = fresh([1024, 1, 1500, 255], lo, hi, param=param)
    check8(case, *run_step(case, step=1, max_norm=0.0, eps=eps)[:3])


@pytest.mark.parametrize("step", [2, 1000])
def test_eps_0_from_a_stored_state(step):
    """Elements whose root fell to the least byte, and ones that had no gradient before."""
    case = Case([2048, 300], 8, grad="f32", seed=3)
    case.grads = case.grad_bits = [spread(n, -60, 0, 7 + i) for i, n in enumerate(case.lens)]
    old = [spread(n, -40, 0, 17 + i) for i, n in enumerate(case.lens)]
    for x in old:
        x[::7] = 0.0
    case.state = [S8.encode(0.1 * x.astype(np.float64), 0.01 * x.astype(np.float64) ** 2) for x in old]
    case.to_device()
    check8(case, *run_step(case, step=step, eps=0.0)[:3])


def test_eps_0_in_a_long_list():
    """Units of a wave of their own, next to a tensor's partial last block."""
    case = fresh([1100 * 1024 + 130, 77], -110, 0)
    check8(case, *run_step(case, step=1, eps=0.0)[:3])
