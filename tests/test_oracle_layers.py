"""The fp64 oracle of token tables and norms against torch's own definitions in
fp64 and against differences."""

import numpy as np
import pytest

from oracle import layers as O

torch = pytest.importorskip("torch")


def test_embedding_and_its_gradient():
    r = np.random.default_rng(0)
    tok = r.integers(-2, 9, 50)
    W, d = r.standard_normal((7, 5)), r.standard_normal((50, 5))
    out = O.embedding(tok, W, 1.5)
    inside = (tok >= 0) & (tok < 7)
    assert (out[~inside] == 0).all()
    assert np.array_equal(out[inside], 1.5 * W[tok[inside]])
    one_hot = np.zeros((50, 7))
    one_hot[np.flatnonzero(inside), tok[inside]] = 1.0
    assert np.allclose(O.embedding_grad(tok, d, 7, 1.5), 1.5 * one_hot.T @ d, rtol=1e-13, atol=1e-13)
    rows, pos = O.token_order(tok, 7)
    assert rows == sorted(tok[inside].tolist()) and sorted(pos) == np.flatnonzero(inside).tolist()
    assert all(tok[p] == k for k, p in zip(rows, pos))
    assert all(a < b for (k, a), (j, b) in zip(zip(rows, pos), list(zip(rows, pos))[1:]) if k == j)


@pytest.mark.parametrize("affine", [False, True])
def test_layer_norm_is_torch_s(affine):
    r = np.random.default_rng(1)
    x, dy = r.standard_normal((6, 33)) * 2 + 1, r.standard_normal((6, 33))
    w, b = (r.standard_normal(33), r.standard_normal(33)) if affine else (None, None)
    t = [None if v is None else torch.from_numpy(v).requires_grad_() for v in (x, w, b)]
    y = torch.nn.functional.layer_norm(t[0], (33,), t[1], t[2], 1e-5)
    got, mean, rstd = O.norm(x, w, b, 1e-5)
    assert np.allclose(got, y.detach().numpy(), rtol=1e-12, atol=1e-12)
    y.backward(torch.from_numpy(dy))
    dx, dw, db = O.norm_grad(dy, x, mean, rstd, w)
    assert np.allclose(dx, t[0].grad.numpy(), rtol=1e-11, atol=1e-12)
    if affine:
        assert np.allclose(dw, t[1].grad.numpy(), rtol=1e-11, atol=1e-12)
        assert np.allclose(db, t[2].grad.numpy(), rtol=1e-11, atol=1e-12)


@pytest.mark.parametrize("rms", [False, True])
def test_norm_gradients_are_the_differences(rms):
    r = np.random.default_rng(2)
    x, dy, w, d_total = r.standard_normal((3, 9)), r.standard_normal((3, 9)), r.standard_normal(9), r.standard_normal((3, 9))

    def loss(x, w, b):
        return (O.norm(x, w, b, 1e-3, rms)[0] * dy).sum() + (x * d_total).sum()

    b = r.standard_normal(9)
    _, mean, rstd = O.norm(x, w, b, 1e-3, rms)
    assert (mean == 0).all() == rms
    for arg, g in enumerate(O.norm_grad(dy, x, mean, rstd, w, d_total, rms)):
        for at in np.ndindex(g.shape):
            val = []
            for e in (1e-6, -1e-6):
                a = [x.copy(), w.copy(), b.copy()]
                a[arg][at] += e
                val.append(loss(*a))
            # central differences: the third derivative's term and the loss's last bits over the step
            assert abs((val[0] - val[1]) / 2e-6 - g[at]) <= 1e-7 * (1 + np.abs(g).max())
