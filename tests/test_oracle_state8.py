"""The 8-bit moments of the oracle pinned: the e4m3 bytes against torch's
float8 type, the rounding against an exhaustive search, blocks and scales
against a direct loop, and the step against torch.optim.AdamW in fp64."""

from fractions import Fraction

import numpy as np
import pytest

from oracle import state8 as S
from oracle import step as O

torch = pytest.importorskip("torch")


def test_bytes_are_torch_float8_e4m3fn():
    t = torch.arange(256, dtype=torch.int16).to(torch.uint8).view(torch.float8_e4m3fn).to(torch.float64).numpy()
    got = S.e4m3_table()
    assert np.array_equal(np.isnan(t), np.isnan(got))
    assert np.array_equal(t[~np.isnan(t)], got[~np.isnan(got)])


def test_rounding_against_exact_search():
    """The nearest of the 253 finite values by exact rational distance, ties
    to the even byte; border values and their neighbours among the inputs."""
    grid = S.e4m3_table()[:127]
    mid = (grid[:-1] + grid[1:]) / 2
    rng = np.random.default_rng(0)
    x = np.concatenate([grid, mid, np.nextafter(mid, 0), np.nextafter(mid, 1e9), rng.random(300) * 460,
                        2.0 ** rng.uniform(-14, 8.8, 300)])
    x = np.concatenate([x, -x])
    got = S.e4m3_encode(x)
    exact = [Fraction(float(v)) for v in grid]
    for value, code in zip(x, got):
        a = abs(Fraction(float(value)))
        best = min(range(127), key=lambda k: (abs(exact[k] - a), k % 2))
        assert code & 0x7F == best, (value, code, best)
        assert (code >= 128) == bool(np.signbit(value))
    assert (S.e4m3_encode([np.nan, np.inf, -np.inf, 465.0]) & 0x7F == S.NAN).all()
    assert S.e4m3_encode([464.0, 448.0]).tolist() == [0x7E, 0x7E]


def test_float32_cast_agrees_away_from_double_rounding():
    x = np.random.default_rng(1).standard_normal(20000).astype(np.float32) * 50
    t = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(t, S.e4m3_encode(x))


@pytest.mark.parametrize("n", [0, 1, 255, 256, 257, 1000])
def test_blocks_and_scales(n):
    rng = np.random.default_rng(n)
    m, v = rng.standard_normal(n) * 1e-4, rng.random(n) ** 8 * 1e-6
    if n > 20:
        v[3:9], m[5] = 0.0, 0.0
    mc, ms, vc, vs = S.encode(m, v)
    assert mc.size == vc.size == n and ms.size == vs.size == -(-n // 256)
    for b in range(ms.size):
        x, r = m[256 * b:256 * b + 256], np.sqrt(v[256 * b:256 * b + 256])
        top = np.float32(np.abs(x).max())
        assert ms[b] == np.float32(float(top) / 448)
        assert abs(vs[b] - r.max() / 448) <= 2.0 ** -22 * vs[b]
        assert (np.abs(S.e4m3_decode(mc[256 * b:256 * b + 256])).max()) == 448
    dm, dv = S.decode(mc, ms, vc, vs)
    spread = np.repeat(ms.astype(np.float64), 256)[:n]
    assert (np.abs(dm - m) <= np.maximum(2.0 ** -4 * np.abs(m) * (1 + 1e-6), 2.0 ** -10 * spread * (1 + 1e-6))).all()
    assert ((dv > 0) == (v > 0)).all()


def test_not_finite_moments_spoil_their_element_only():
    m, v = np.linspace(-1, 1, 300), np.linspace(0, 2, 300)
    clean = S.encode(m, v)
    bad_m, bad_v = m.copy(), v.copy()
    bad_m[7], bad_v[9], bad_m[299], bad_v[11] = np.nan, np.inf, -np.inf, -1.0
    got = S.encode(bad_m, bad_v)
    for k, holes in ((0, [7, 299]), (2, [9, 11])):
        same = np.ones(300, bool)
        same[holes] = False
        assert (got[k][holes] & 0x7F == S.NAN).all()
        assert np.array_equal(got[k][:256][same[:256]], clean[k][:256][same[:256]])
    assert got[1][0] == clean[1][0] and got[3][0] == clean[3][0]


def test_step_is_adamw_on_the_decoded_state():
    n, step = 700, 12
    rng = np.random.default_rng(3)
    hp = O.AdamWHParams(lr=3e-3, weight_decay=0.1)
    state = S.encode(rng.standard_normal(n) * 1e-2, rng.random(n) * 1e-3)
    m, v = S.decode(*state)
    p, g = rng.standard_normal(n), rng.standard_normal(n) * 0.1
    w = torch.nn.Parameter(torch.from_numpy(p.copy()))
    opt = torch.optim.AdamW([w], lr=hp.lr, weight_decay=hp.weight_decay, foreach=False)
    opt.state[w] = {"step": torch.tensor(float(step - 1)), "exp_avg": torch.from_numpy(m.copy()),
                    "exp_avg_sq": torch.from_numpy(v.copy())}
    w.grad = torch.from_numpy(0.7 * g)
    opt.step()
    p1, m1, v1, codes = S.adamw8_step(g, p, *state, step, hp, 0.7)
    assert np.allclose(p1, w.detach().numpy(), rtol=1e-12, atol=1e-15)
    assert np.allclose(m1, opt.state[w]["exp_avg"].numpy(), rtol=1e-12, atol=1e-18)
    assert np.allclose(v1, opt.state[w]["exp_avg_sq"].numpy(), rtol=1e-12, atol=1e-18)
    for a, b in zip(codes, S.encode(m1, v1)):
        assert np.array_equal(a, b)


def test_zero_state_is_zero_moments():
    z8, zs = np.zeros(300, np.uint8), np.zeros(2, np.float32)
    m, v = S.decode(z8, zs, z8, zs)
    assert not m.any() and not v.any()
    mc, ms, vc, vs = S.encode(m, v)
    assert not mc.any() and not vc.any() and np.isfinite(ms).all() and np.isfinite(vs).all()
