"""The 8-bit step where a second moment passes fp32: the element's step is zero
and its byte the NaN, and its neighbours are what they are without it."""

import numpy as np
import pytest

import state8_codes
from oracle import state8 as S8
from oracle import step as O
from tensor_lists import Case
from test_gpu_tensors import run_step

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("param", ["bf16", "f32"])
def test_a_second_moment_beyond_fp32(param):
    case = Case([600, 300], 8, param, "f32", seed=60)
    huge = {7: 1e25, 300: -3e30, 511: 3e38}
    for k, x in huge.items():
        case.grads[0][k] = x
    case.to_device()
    (hp,), (step,), coef, _ = run_step(case, max_norm=0.0)
    case.check_guards()
    got = {k: a.tensors() for k, a in case.A.items()}
    masters = got["master"] if "master" in got else got["param"]
    at, rest = np.array(list(huge)), np.setdiff1d(np.arange(600), list(huge))
    # decay only: lr * wd rounded once, the product within the fused multiply-add
    want = case.master[0][at].astype(np.float64) * (1 - hp.lr * hp.weight_decay)
    assert (np.abs(masters[0][at] - want) <= 2 * 2.0 ** -24 * np.abs(want)).all()
    p, m1, v1, _ = S8.adamw8_step(case.grads[0], case.master[0], *case.state[0], step, hp, coef)
    assert (np.abs(masters[0][rest] - p[rest]) <= S8.update_bound(case.master[0], m1, v1, step, hp)[rest]).all()
    assert (got["v"][0][at] & 0x7F == S8.NAN).all() and np.isfinite(masters[0]).all()
    with np.errstate(over="ignore"):
        v1 = np.where(np.isinf(v1.astype(np.float32)), np.inf, v1)       # as the state takes it
    state8_codes.check([got[k][0] for k in ("m", "m_scale", "v", "v_scale")], m1, v1,
                       state8_codes.step_slack(case.grads[0], *case.state[0], hp, coef))
