"""Token tables and norms in fp64, from their definitions, one row at a time
where that is plainest. Arrays are numpy; a token outside the table reads as
zeros and has no gradient."""

from __future__ import annotations

import numpy as np


def embedding(tokens, table, scale=1.0):
    table = np.asarray(table, np.float64)
    out = np.zeros((len(tokens), table.shape[1]))
    for t, k in enumerate(tokens):
        if 0 <= k < len(table):
            out[t] = scale * table[k]
    return out


def embedding_grad(tokens, d_out, rows, scale=1.0):
    d_out = np.asarray(d_out, np.float64)
    grad = np.zeros((rows, d_out.shape[1]))
    for t, k in enumerate(tokens):
        if 0 <= k < rows:
            grad[k] += d_out[t]
    return scale * grad


def token_order(tokens, rows):
    """The rows and positions of the tokens inside the table, sorted by row, then by position."""
    at = sorted((int(k), t) for t, k in enumerate(tokens) if 0 <= k < rows)
    return [k for k, _ in at], [t for _, t in at]


def norm(x, weight=None, bias=None, eps=1e-5, rms=False):
    """(y, mean, rstd) of the rows of x; mean is zero with rms."""
    x = np.asarray(x, np.float64)
    mean = np.zeros(len(x)) if rms else x.mean(1)
    dev = x - mean[:, None]
    with np.errstate(divide="ignore", invalid="ignore"):
        rstd = 1.0 / np.sqrt((dev * dev).mean(1) + eps)
        y = dev * rstd[:, None]
    if weight is not None:
        y = y * np.asarray(weight, np.float64)
    if bias is not None:
        y = y + np.asarray(bias, np.float64)
    return y, mean, rstd


def norm_grad(d_y, x, mean, rstd, weight=None, d_total=None, rms=False):
    """(d_x, d_weight, d_bias) from the statistics of the forward pass."""
    d_y, x = np.asarray(d_y, np.float64), np.asarray(x, np.float64)
    rstd = np.asarray(rstd, np.float64)[:, None]
    xh = (x if rms else x - np.asarray(mean, np.float64)[:, None]) * rstd
    g = d_y if weight is None else d_y * np.asarray(weight, np.float64)
    d_x = g - xh * (g * xh).mean(1, keepdims=True)
    if not rms:
        d_x = d_x - g.mean(1, keepdims=True)
    d_x = d_x * rstd
    if d_total is not None:
        d_x = d_x + np.asarray(d_total, np.float64)
    return d_x, (d_y * xh).sum(0), d_y.sum(0)
