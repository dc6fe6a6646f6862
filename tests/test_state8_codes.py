"""The check of 8-bit states itself, on the host: it takes what the definition
gives, and finds a wrong scale, and a wrong byte whatever its block's scale."""

import numpy as np
import pytest

import state8_codes
from oracle import state8 as S8
from oracle import step as O
from test_gpu_tensors import check_codes


def drawn(n, seed=0):
    rng = np.random.default_rng(seed)
    return rng.standard_normal(n) * 1e-3, (rng.standard_normal(n) * 1e-3) ** 2


@pytest.mark.parametrize("n", [0, 1, 255, 256, 257, 4099])
def test_the_definition_passes(n):
    m, v = drawn(n)
    assert state8_codes.check(S8.encode(m, v), m, v) == 0
    off = 16 * 2.0 ** -53
    assert state8_codes.check(S8.encode(m * (1 + off / 2), v * (1 - off / 2)), m, v, (off * np.abs(m), off * v)) == 0


def test_moments_that_are_not_finite():
    m, v = drawn(300)
    m[3], m[4], v[5], v[6], v[7], v[8] = np.nan, np.inf, np.nan, np.inf, -1.0, -0.0
    assert state8_codes.check(S8.encode(m, v), m, v) == 0


def test_a_steps_slack_holds_another_order():
    """The same step with fused products, in another order."""
    hp, coef = O.AdamWHParams(), 0.37
    rng = np.random.default_rng(3)
    m, v = drawn(5000, 3)
    state, g = S8.encode(m, v), (rng.standard_normal(5000) * 1e-3).astype(np.float32)
    _, m1, v1, _ = S8.adamw8_step(g, np.zeros(5000), *state, 3, hp, coef)
    dm, dv = S8.decode(*state)
    ml, gl = dm.astype(np.longdouble), g.astype(np.longdouble) * np.longdouble(coef)
    m2 = (np.longdouble(hp.beta1) * ml + (1 - np.longdouble(hp.beta1)) * gl).astype(np.float64)
    v2 = (np.longdouble(hp.beta2) * dv + (1 - np.longdouble(hp.beta2)) * gl * gl).astype(np.float64)
    state8_codes.check(S8.encode(m2, v2), m1, v1, state8_codes.step_slack(g, *state, hp, coef))


@pytest.mark.parametrize("kind", ["scale", "bytes", "bytes of a block with the scale's neighbour"])
@pytest.mark.parametrize("moment", [0, 1])
def test_mistakes_are_found(kind, moment):
    m, v = drawn(4099)
    good = S8.encode(m, v)
    slack = 16 * 2.0 ** -53 * np.abs(m), 16 * 2.0 ** -53 * v
    bad = [x.copy() for x in good]
    if kind != "bytes":
        bad[2 * moment + 1] = np.nextafter(bad[2 * moment + 1], np.float32(0))
    if kind != "scale":
        bad[2 * moment][:] = 0
    if kind != "bytes":       # what the older check lets through: it looks at no byte of such a block
        check_codes(bad, good, "tensor") if good[0].size <= 25600 else None
    with pytest.raises(AssertionError, match="scales" if kind != "bytes" else "bytes"):
        state8_codes.check(bad, m, v, slack)


def test_bytes_are_held_to_the_scale_that_was_stored():
    """A maximum within the slack of a border: its other scale is taken, with the bytes that belong to it only."""
    x = np.float32(1e-3)
    border = (float(x) + float(np.nextafter(x, np.float32(1)))) / 2
    m = np.linspace(-0.9e-3, 0.9e-3, 256)
    m[17] = border * (1 - 2.0 ** -53)
    v = np.full(256, 1e-6)
    slack = 4 * 2.0 ** -53 * np.abs(m), np.zeros(256)
    above = m.copy()
    above[17] = border * (1 + 2.0 ** -52)
    other = S8.encode(above, v)
    assert other[1][0] != S8.encode(m, v)[1][0]
    assert state8_codes.check(other, m, v, slack) == 1
    bad = [c.copy() for c in other]
    bad[0][40] ^= 1
    with pytest.raises(AssertionError, match="bytes"):
        state8_codes.check(bad, m, v, slack)
    with pytest.raises(AssertionError, match="scales"):
        state8_codes.check(other, m, v)
