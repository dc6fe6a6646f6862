"""The tensor-list step with moments in 8 bits, in plain numpy float64: the
e4m3 rounding, blocks with their scales, and AdamW on the state they hold.

The pages keep the optimizer state at K = 12 bytes per parameter in fp32
("第 5 课：ZeRO 与 FSDP", section 2) and give no 8-bit form, so the definition is
this library's own: m and sqrt(v) as OCP e4m3 values with one fp32 scale per
256 consecutive elements of a tensor (include/zero_tensors.h). The rest is
AdamW as in ``oracle.step``. Rounding to nearest keeps a root that moves by
less than half a step of its byte: one update is AdamW's on the state it finds,
a chain of them only up to beta2 = 0.95 or so.
"""

from __future__ import annotations

import math

import numpy as np

from .step import AdamWHParams, adamw_f64

BLOCK = 256
E4M3_MAX = 448.0
LEAST_MAX = 2.0 ** -100       # smallest maximum a scale of m is formed from
LEAST_ROOT = 2.0 ** -63       # the same for the roots: below, the maximum's square is subnormal in fp32
NAN = 0x7F


def e4m3_table() -> np.ndarray:
    """Values of the 256 bytes: sign, 4 exponent bits (bias 7), 3 fraction
    bits; no infinities, S.1111.111 is NaN."""
    b = np.arange(256)
    e, f = (b >> 3) & 15, b & 7
    mag = np.where(e == 0, f * 2.0 ** -9, (8 + f) * 2.0 ** (e - 10.0))
    mag[(b & 0x7F) == NAN] = np.nan
    return np.where(b < 128, mag, -mag)


_TABLE = e4m3_table()


def e4m3_decode(codes) -> np.ndarray:
    return _TABLE[np.asarray(codes, np.uint8)]


def e4m3_encode(x) -> np.ndarray:
    """Bytes of the nearest e4m3 values (ties to even) of float64 values; what
    rounds beyond 448, and NaN, give the NaN byte."""
    x = np.asarray(x, np.float64)
    a = np.abs(x)
    grid = _TABLE[:127]
    mid = (grid[:-1] + grid[1:]) / 2                       # exact
    k = np.searchsorted(mid, a, side="left")               # borders below a: the value at a border is the lower one
    tie = (k < 126) & (mid[np.minimum(k, 125)] == a)
    k = k + (tie & (k % 2 == 1))                           # a tie goes to the even byte
    k = np.where(np.isnan(a) | (a > 464.0), NAN, k)
    return (k + np.where(np.signbit(x) & ~np.isnan(x), 128, 0)).astype(np.uint8)


def _blocks(x):
    """Rows of 256 (the last one padded with zeros)."""
    return np.pad(x, (0, -x.size % BLOCK)).reshape(-1, BLOCK)


def _top(x):
    """fp32 maximum of each row's finite values (0 if none is positive)."""
    with np.errstate(over="ignore"):
        a = x.astype(np.float32)
    return np.where(np.isfinite(a), a, np.float32(0)).max(axis=1).astype(np.float32)


def encode(m, v):
    """(m bytes, m scales, v bytes, v scales) of float64 moments of one tensor."""
    n = np.asarray(m).size
    if n == 0:
        return np.zeros(0, np.uint8), np.zeros(0, np.float32), np.zeros(0, np.uint8), np.zeros(0, np.float32)
    mb, vb = _blocks(np.asarray(m, np.float64)), _blocks(np.asarray(v, np.float64))
    tops = [_top(np.abs(mb)), np.sqrt(_top(vb))]                   # fp32 square root, correctly rounded
    tops = [np.maximum(t, np.float32(least)) for t, least in zip(tops, (LEAST_MAX, LEAST_ROOT))]
    up = [(np.float32(E4M3_MAX) / t).astype(np.float64)[:, None] for t in tops]
    with np.errstate(invalid="ignore"):
        root = np.sqrt(vb) * up[1]
        mc = e4m3_encode(mb * up[0])
        vc = e4m3_encode(np.where(vb > 0, np.maximum(root, 2.0 ** -9), root))
    scales = [(t / np.float32(E4M3_MAX)).astype(np.float32) for t in tops]
    return mc.reshape(-1)[:n], scales[0], vc.reshape(-1)[:n], scales[1]


def decode(m_codes, m_scale, v_codes, v_scale):
    """float64 moments that the bytes and scales of one tensor stand for."""
    n = np.asarray(m_codes).size
    spread = lambda s: np.repeat(np.asarray(s, np.float64), BLOCK)[:n]  # noqa: E731
    root = e4m3_decode(v_codes) * spread(v_scale)
    return e4m3_decode(m_codes) * spread(m_scale), root * root


def adamw8_step(grad, master, m_codes, m_scale, v_codes, v_scale, step: int, hp: AdamWHParams, coef: float):
    """One tensor's step on the 8-bit state. ``grad``: the gradient's values.
    Returns (master' in float64, m', v' in float64 before they are rounded to
    8 bits, the new bytes and scales as ``encode`` gives them)."""
    m, v = decode(m_codes, m_scale, v_codes, v_scale)
    g = coef * np.asarray(grad, np.float64)
    p1, m1, v1 = adamw_f64(np.asarray(master, np.float64), m, v, g, step, hp)
    return p1, m1, v1, encode(m1, v1)


def update_bound(master, m1, v1, step: int, hp: AdamWHParams):
    """|master - p'| allowed to an fp32 evaluation of the update from m1, v1,
    in units of 2^-24 (a rounding to nearest is 1, a hardware square root or
    reciprocal within one unit in the last place is 2, and what is under a
    square root counts half):

    of the master: the decayed value 1, its constant under 1, the result 1;
    of the step: its constant 1, m1 1, the reciprocal 2, the quotient 1, the
    result 1; of the denominator under it: v1 1/2, the square of 448 / largest
    root 1/2, their product 1/2, the square root 2, 448 / root and root / 448
    one each, their product with the root 1, the bias constant or eps 1, the
    sum 1. 6 + 8.5 = 14.5, and 1/2 for the products of these errors."""
    bias1, bias2 = 1.0 - hp.beta1 ** step, 1.0 - hp.beta2 ** step
    move = np.abs(hp.lr / bias1 * m1 / (np.sqrt(v1) / math.sqrt(bias2) + hp.eps))
    return 2.0 ** -24 * (3 * np.abs(np.asarray(master, np.float64)) + 15 * move)
