"""Inputs and tolerances of the token-table and norm tests.

Tolerances are bounds, not measurements. u = 2^-24 is half a step of fp32, h half
a step of the stored type (2^-8 for bf16, u for fp32), both relative to the value.
A sum of values taken in fp32 with at most k additions on any value's way to the
result is off by at most k u times the sum of the magnitudes, to first order; the
second orders are covered by SLACK. What a product or a difference adds is named
where it is used."""

import numpy as np
import torch

from oracle import layers as O

U = 2.0 ** -24
SLACK = 1.05
TINY = 2.0 ** -126         # results below the normal numbers are not held to a relative bound
DEV = "cuda"


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def np64(t):
    return None if t is None else t.detach().to(torch.float64).cpu().numpy()


def close(got, want, bound, what):
    got, want = np64(got), np.asarray(want)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    err = np.abs(got - want)
    bad = ~(err <= SLACK * bound + TINY)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} off; first {np.argwhere(bad)[:3].tolist()}: got "
                           f"{got[bad][:3]}, want {want[bad][:3]}, bound {np.broadcast_to(bound, bad.shape)[bad][:3]}")


def generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def normal(gen, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=gen, device=DEV) * std).to(dtype)


def rows_of(t, stride, fill=float("nan")):
    """t's values in an array whose rows are `stride` elements apart; what lies between them is `fill`."""
    n, dim = t.shape
    whole = torch.full((n, stride), fill, dtype=t.dtype, device=t.device)
    whole[:, :dim] = t
    return whole[:, :dim], whole


def shifted(t, by):
    """t's values, starting `by` elements behind a 16-byte boundary."""
    whole = torch.full((t.numel() + by,), float("nan"), dtype=t.dtype, device=t.device)
    whole[by:] = t.flatten()
    return whole[by:].view(t.shape)


def draw_tokens(n, rows, seed, kind="mixed", dtype=torch.int64):
    """mixed: frequent and rare ones, some outside the table; same: one row; distinct: all different as far as
    the table has rows; none: all outside."""
    r = np.random.default_rng(seed)
    if kind == "same":
        t = np.full(n, rows // 2)
    elif kind == "distinct":
        t = r.permutation(max(n, rows))[:n] % rows
    elif kind == "none":
        t = np.full(n, -1)
    else:
        t = np.minimum((rows * r.random(n) ** 4).astype(np.int64), rows - 1)
        t = r.permutation(rows)[t]
        t[r.random(n) < 0.15] = -1
        t[r.random(n) < 0.05] = rows           # one past the end
        if n > 3:
            t[n // 2] = np.iinfo(np.int32).min if dtype == torch.int32 else np.iinfo(np.int64).min
            t[n // 3] = np.iinfo(np.int32).max if dtype == torch.int32 else (1 << 32)      # its low half is row 0
    return torch.from_numpy(t).to(dtype).to(DEV)


def embedding_grad_want(tokens, d_out, rows, scale, old=None):
    """The whole table's gradient and, per element, the bound without the store's rounding: c terms are
    c - 1 additions, then the scale's product (with `old` one rounding for both, as an fma)."""
    tok, d = tokens.flatten().cpu().numpy(), np64(d_out)
    want = O.embedding_grad(tok, d, rows, scale)
    size = O.embedding_grad(tok, np.abs(d), rows, abs(scale))
    count = np.zeros((rows, 1))
    for k in tok:
        if 0 <= k < rows:
            count[k] += 1
    bound = count * U * size
    if old is not None:
        want = want + np64(old).reshape(want.shape)
    return want, bound + U * np.abs(want)


def sum_depth(dim):
    """Additions on a value's way into a row's sum: up to 32 in its thread (or one vector of 8 for every 4096
    elements of a long row), 6 over the wave, 16 over the waves."""
    return 64 + dim / 512


def norm_bounds(s, weight, bias, eps, rms, dtype):
    """Of y, mean and rstd for the rows `s` that the kernel reads."""
    s = np64(s)
    y, mean, rstd = O.norm(s, np64(weight), np64(bias), eps, rms)
    dim, k = s.shape[1], sum_depth(s.shape[1])
    w = np.ones(dim) if weight is None else np.abs(np64(weight))
    var = ((s - mean[:, None]) ** 2).mean(1)
    d_mean = np.zeros(len(s)) if rms else k * U * np.abs(s).mean(1) + U * np.abs(mean)
    # the squares after a mean that is off by d_mean: the deviations' mean is zero, so their squares' is off by d_mean^2
    d_var = d_mean ** 2 + (k + 4) * U * (var + d_mean ** 2)
    with np.errstate(divide="ignore", invalid="ignore"):
        rel = 0.5 * (d_var + 2 * U * (var + eps)) / (var + eps) + 2 * U     # sum with eps, root, quotient
    xh = np.abs(s - mean[:, None]) * rstd[:, None]
    d_y = w * rstd[:, None] * d_mean[:, None] + w * xh * (rel[:, None] + 3 * U) + U * np.abs(y)
    return (y, mean, rstd), (d_y + half_step(dtype) * (np.abs(y) + d_y), d_mean, rel * rstd)


def norm_grad_want(d_y, x, mean, rstd, weight, d_total, rms, dtype):
    """d_x, d_weight, d_bias and their bounds, of the last two without the store's rounding."""
    dy, xs, m, r = np64(d_y), np64(x), np64(mean), np64(rstd)[:, None]
    want = O.norm_grad(dy, xs, m, r[:, 0], np64(weight), np64(d_total), rms)
    dim, n = xs.shape[1], len(xs)
    w = np.ones(dim) if weight is None else np64(weight)
    k = sum_depth(dim)
    dev = xs if rms else xs - m[:, None]
    xh, g = np.abs(dev) * r, np.abs(dy * w)
    c1 = np.abs((dy * w * dev * r).mean(1, keepdims=True))
    c0 = 0.0 if rms else np.abs((dy * w).mean(1, keepdims=True))
    e0 = 0.0 if rms else (k + 2) * U * g.mean(1, keepdims=True)           # g's product, the sum, the quotient
    e1 = (k + 5) * U * (g * xh).mean(1, keepdims=True)                    # also x - mean, times rstd, the product
    # the product g, minus c0, the fma with xh (off by 2 u) and c1, the fma with rstd
    inner = U * g + e0 + U * (g + c0) + xh * e1 + 2 * U * xh * c1 + U * (g + c0 + xh * c1)
    b_x = r * inner + U * np.abs(want[0])
    b_x = b_x + half_step(dtype) * (np.abs(want[0]) + b_x)
    # a column's sum: rows in turn in a block, then the blocks'; never more than n additions
    kn = min(n, 128 + n / 64)
    b_w = (kn + 3) * U * (np.abs(dy) * xh).sum(0)
    b_b = kn * U * np.abs(dy).sum(0)
    return want, (b_x, b_w, b_b)


def stored(bound, want, dtype):
    """The bound with the rounding to the stored type."""
    return bound + half_step(dtype) * (np.abs(want) + bound)
