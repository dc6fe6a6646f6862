"""Norms of rows whose mean is far larger than their deviation, where the rounding
of an fp32 mean is itself a deviation.

The bounds, with u = 2^-24 and k additions on a value's way into a row's sum: the
first mean is off by at most D = k u mean|s| + u |mean|. The deviations from it sum to
dim times its error, up to E = (k + 2) u (mean|dev| + D) a deviation (their own
rounding, the sum's, the quotient's). Taken off again, that leaves a deviation off by
E + u (2 |dev| + D), and the squares' sum, less the square of the correction, off by
(k + 5) u (var + D^2) + 2 D E + E^2 + u (D + E)^2. Taken off as a shift of the normalised
values, it is rounded once more, by u D at most. The stored mean is off by E and its
rounding. D enters in second order only.

A row whose mean is not above sqrt(var + eps) keeps its first mean. There E is D, the
squares' sum is off by D^2, which the terms above cover, and since mean|s| <= |mean| +
mean|dev| <= 2 sqrt(var + eps), D / sqrt(var + eps), what y is off by for a weight of one,
is (2 k + 1) u at most: the rounding of a sum of such rows, whatever its method."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from fsdp_sharded_mixed_zero_amd import layers

import layer_cases as C  # noqa: E402
from layer_cases import DEV, U, close, generator, half_step, normal  # noqa: E402
from oracle import layers as O  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32
EPS = 1e-5


def bounds(s, weight, bias, dtype):
    """y, mean and rstd of the rows that the kernel reads, and their bounds."""
    s, w = C.np64(s), np.abs(C.np64(weight))
    y, mean, rstd = O.norm(s, C.np64(weight), C.np64(bias), EPS)
    k, dev = C.sum_depth(s.shape[1]), np.abs(s - mean[:, None])
    var = (dev ** 2).mean(1)
    D = k * U * np.abs(s).mean(1) + U * np.abs(mean)
    E = (k + 2) * U * (dev.mean(1) + D)
    near = np.abs(mean) <= 1.001 * np.sqrt(var + EPS)        # 1.001: the decision is made on rounded values
    E = np.where(near, np.maximum(E, D), E)
    d_var = (k + 5) * U * (var + D ** 2) + 2 * D * E + E ** 2 + U * (D + E) ** 2
    rel = 0.5 * (d_var + 2 * U * (var + EPS)) / (var + EPS) + 2 * U          # sum with eps, root, quotient
    off = (E + 2 * U * D)[:, None] + 2 * U * dev
    r = rstd[:, None]
    d_y = w * r * off + w * dev * r * (rel[:, None] + 2 * U) + U * np.abs(y)
    return (y, mean, rstd), (d_y + half_step(dtype) * (np.abs(y) + d_y), E + U * np.abs(mean), rel * rstd)


def check(x, dtype, residual=None):
    n, dim = x.shape
    gen = generator(dim + n)
    w, b = normal(gen, dim), normal(gen, dim)
    y, mean, rstd = torch.empty_like(x), torch.empty(n, device=DEV), torch.empty(n, device=DEV)
    total = None if residual is None else torch.empty_like(x)
    layers.zero_norm(x, y, mean, rstd, weight=w, bias=b, eps=EPS, residual=residual, total=total)
    want, bound = bounds(x if total is None else total, w, b, dtype)
    for got, v, e, what in zip((y, mean, rstd), want, bound, ("y", "mean", "rstd")):
        close(got, v, e, what)


# one vector or less, a part of a wave, a wave, several, several waves, the rows that are read three times
DIMS = [1, 2, 7, 33, 129, 777, 1111, 1600, 4099, 8192, 12001, 16385, 40000, 70001]


@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("value", [1000.1, -10000.1, 0.3, 3e-4])
def test_constant_rows(dim, value):
    """A row without deviation gives the bias, however its mean is rounded."""
    for n in (2, 1030) if 500 < dim < 1100 else (2,):
        check(torch.full((n, dim), value, device=DEV), F32)


@pytest.mark.parametrize("dim", DIMS)
def test_constant_rows_of_a_residual_and_of_bf16(dim):
    x = torch.full((3, dim), 700.3, device=DEV)
    check(x, F32, residual=torch.full_like(x, 299.9))
    check(x.to(BF16), BF16, residual=x.to(BF16) * -3)


@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_means_far_larger_than_deviations(dim, dtype):
    """1e4 times the deviation in fp32, 100 times in bf16, each row with another mean."""
    gen = generator(dim)
    far = 1e4 if dtype == F32 else 100.0
    for n in (5, 1030) if 500 < dim < 1100 else (5,):
        x = (normal(gen, n, dim) + far * (1.0 + torch.arange(n, device=DEV)[:, None] / 7)).to(dtype)
        check(x, dtype)
        check(x, dtype, residual=(normal(gen, n, dim) * far).to(dtype))


@pytest.mark.parametrize("dim", [3, 96, 1500, 9000, 40000])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_bad_values_keep_their_means(dim, dtype):
    """A row with an infinity has an infinite mean, one with a NaN none; the others are as without them."""
    x = normal(generator(dim), 5, dim, dtype=dtype)
    clean = x.clone()
    x[1, 0], x[2, dim - 1], x[3, dim // 2] = float("inf"), -float("inf"), float("nan")
    y, mean, rstd = torch.empty_like(x), torch.empty(5, device=DEV), torch.empty(5, device=DEV)
    layers.zero_norm(x, y, mean, rstd)
    assert mean[1] == float("inf") and mean[2] == -float("inf") and torch.isnan(mean[3])
    assert torch.isnan(rstd[1:4]).all() and torch.isnan(y[1:4]).all()
    alone, m, r = torch.empty_like(x), torch.empty_like(mean), torch.empty_like(rstd)
    layers.zero_norm(clean, alone, m, r)
    for a, b in ((y, alone), (mean, m), (rstd, r)):
        assert torch.equal(a[[0, 4]], b[[0, 4]])


@pytest.mark.parametrize("dim", [5, 33, 100, 129, 200, 300, 777, 1600, 20000])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_far_and_near_means_side_by_side(dim, dtype):
    """Rows that keep their first mean between rows that do not, several of them in a wave: each as if alone."""
    n = 37
    x = normal(generator(dim), n, dim)
    x[::3] += 1e4 if dtype == F32 else 100.0
    x[1::6] = 1000.1
    x = x.to(dtype)
    y, mean, rstd = torch.empty_like(x), torch.empty(n, device=DEV), torch.empty(n, device=DEV)
    layers.zero_norm(x, y, mean, rstd)
    one = torch.ones(dim, device=DEV)
    want, bound = bounds(x, one, torch.zeros(dim, device=DEV), dtype)
    for got, v, e, what in zip((y, mean, rstd), want, bound, ("y", "mean", "rstd")):
        close(got, v, e, what)
    for k in range(n):
        y1, m1, r1 = torch.empty_like(x[:1]), torch.empty(1, device=DEV), torch.empty(1, device=DEV)
        layers.zero_norm(x[k:k + 1], y1, m1, r1)
        assert torch.equal(y1[0], y[k]) and torch.equal(m1[0], mean[k]) and torch.equal(r1[0], rstd[k])
