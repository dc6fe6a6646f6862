"""The 8-bit second moment over many steps, on the host: which changes of a
root its byte can follow, and how far it stays from AdamW's. The form rounds
to nearest, so a root that moves by less than half a step of its byte comes
back as it was."""

import numpy as np
import pytest

from oracle import state8 as S8
from oracle import step as O

GRID = S8.e4m3_table()[:127]


def one_step(codes, x, beta2):
    """The bytes after a step with g^2 = x * v, in blocks whose largest root stays as it is."""
    n = codes.size
    assert n < S8.BLOCK
    codes = np.append(codes, 0x7E).astype(np.uint8)
    scale = np.float32(2.0 ** -20)                     # 448 scales are exact in fp32, and so is their square's root
    v = (GRID[codes] * float(scale)) ** 2
    g2 = np.append(np.broadcast_to(x, n), 1.0) * v
    out = S8.encode(np.zeros(n + 1), beta2 * v + (1 - beta2) * g2)
    assert abs(out[3][0] / scale - 1) <= 2.0 ** -22
    return out[2][:n]


def test_what_a_step_has_to_change():
    """Half a step of e4m3 is 1/30 to 1/16 of a value of 2^-6 scales or more:
    with beta2 = 0.999 a gradient whose square is under 68 times v leaves
    every byte as it is, and one of over 131 times v raises them."""
    codes = np.arange(1, 0x7E)
    normal = codes >= 8
    for x in (0.0, 0.5, 1.0, 10.0, 68.0):
        assert np.array_equal(one_step(codes, x, 0.999), codes), x
    # sqrt(0.999 + 0.001 x) = 1 + 1/30 at x = 68.8, 1 + 1/16 at 129.9
    up = one_step(codes[normal], 131.0, 0.999)
    assert (up > codes[normal]).all()


@pytest.mark.parametrize("beta2,falls", [(0.9, True), (0.935, True), (0.94, False), (0.95, False), (0.999, False)])
def test_when_a_root_falls_by_itself(beta2, falls):
    """Without a gradient a root goes down by 1 - sqrt(beta2) of itself; the
    nearest border below a byte is 1/32 of it away. Only under
    beta2 = (31/32)^2 = 0.938 does any byte of 2^-6 scales or more change."""
    codes = np.arange(8, 0x7E)
    now = one_step(codes, 0.0, beta2)
    assert (now < codes).any() == falls
    assert falls or np.array_equal(now, codes)


def simulate(beta2, settle, after, change, n=2048, spread=1.0, seed=0, beta1=0.9):
    """Stored root over AdamW's, for n elements whose gradients are normal, of
    sizes exp(spread * N(0, 1)), from the second moment that they have in the
    mean: ``settle`` steps, then every other element's gradients times
    ``change`` for ``after`` more."""
    rng = np.random.default_rng(seed)
    size = np.exp(spread * rng.standard_normal(n))
    v = size ** 2
    hp = O.AdamWHParams(beta1=beta1, beta2=beta2)
    state, p = S8.encode(np.zeros(n), v), np.zeros(n)
    for t in range(settle + after):
        if t == settle:
            size = size * np.where(np.arange(n) % 2 == 0, change, 1.0)
        g = rng.standard_normal(n) * size
        _, _, _, state = S8.adamw8_step(g, p, *state, t + 1, hp, 1.0)
        v = beta2 * v + (1 - beta2) * g * g
    return np.sqrt(S8.decode(*state)[1] / v)


@pytest.mark.parametrize("change", [1.0, 0.1, 4.0])
@pytest.mark.parametrize("beta2", [0.9, 0.95])
def test_up_to_beta2_0_95_the_roots_follow(beta2, change):
    """98 of 100 roots within 0.8 to 1.4 times AdamW's, every group's median within 10 %."""
    r = simulate(beta2, 200, 400, change)
    low, high = np.percentile(r, [1, 99])
    assert 0.8 <= low and high <= 1.4
    for half in (r[::2], r[1::2]):
        assert 0.9 <= np.median(half) <= 1.1


def test_at_beta2_0_999_they_do_not():
    """The limit that the header states: roots stay where their block's largest
    one takes them. Ten times smaller gradients leave them several times too
    large, and so do larger gradients of their neighbours."""
    r = simulate(0.999, 300, 2500, 0.1)
    assert np.median(r[::2]) > 2.0
    r = simulate(0.999, 300, 2500, 4.0)
    assert np.median(r[1::2]) > 1.5
