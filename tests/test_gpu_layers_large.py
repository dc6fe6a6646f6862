"""Token tables and norms beyond 32-bit offsets, at the most tokens a call takes,
and over more rows than one launch."""

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from fsdp_sharded_mixed_zero_amd import layers  # noqa: E402
import layer_cases as C  # noqa: E402
from layer_cases import DEV, generator, normal  # noqa: E402
from oracle import layers as O  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32
FAR = (1 << 31) + 24            # elements between two rows: the third begins beyond 2^32


@pytest.fixture(autouse=True)
def release():
    yield
    torch.cuda.empty_cache()


def order_of(tokens, rows):
    order = torch.empty(layers.zero_token_order_bytes(tokens.numel(), rows) // 4, dtype=torch.int32, device=DEV)
    layers.zero_token_order(tokens, rows, order)
    return order


@pytest.mark.parametrize("ids", [torch.int32, torch.int64])
@pytest.mark.parametrize("n,rows", [(229377, 50257), (300001, 1009), (1 << 20, 16777215), (16777215, 32000)])
def test_order_of_many_tokens(n, rows, ids):
    g = generator(n)
    tokens = (torch.rand(n, generator=g, device=DEV) ** 3 * (rows + 1)).to(ids) - 1      # some outside
    order = order_of(tokens, rows)
    up = (n + 7) // 8 * 8 + 8
    row, pos = order[:n], order[up:up + n].long()
    live = int((tokens >= 0).sum())
    assert (row[live:] == rows).all() and (row[:live] < rows).all()
    row, pos = row[:live], pos[:live]
    assert torch.equal(tokens[pos].int(), row)
    step = row[1:] - row[:-1]
    assert (step >= 0).all()
    assert (pos[1:] > pos[:-1])[step == 0].all()
    assert len(torch.unique(pos)) == live


def test_embedding_in_a_table_beyond_32_bits():
    rows, dim = 1_200_000, 4096             # 4.9e9 elements
    table = torch.empty(rows, dim, dtype=BF16, device=DEV)
    at = torch.tensor([0, 7, 524288, 1048576, 1048577, rows - 1], device=DEV)
    table[at] = normal(generator(1), 6, dim, dtype=BF16)
    tokens = torch.cat([at.flip(0), at, torch.tensor([rows, -1], device=DEV)])
    out = torch.empty(14, dim, dtype=BF16, device=DEV)
    layers.zero_embedding(tokens, table, out)
    assert torch.equal(out[:6], table[at.flip(0)]) and torch.equal(out[6:12], table[at]) and (out[12:] == 0).all()
    # its whole gradient, and a part that begins beyond 2^32
    d_out = normal(generator(2), 14, dim, dtype=BF16)
    order = order_of(tokens, rows)
    ws = torch.empty(layers.zero_embedding_grad_workspace_bytes(14, dim) // 4, device=DEV)
    grad = table.fill_(1.0)
    layers.zero_embedding_grad(order, rows, d_out, grad.view(-1), ws)
    want = (d_out[:6].flip(0).float() + d_out[6:12].float()).to(BF16)
    assert torch.equal(grad[at], want)
    grad[at] = 0
    assert int(torch.count_nonzero(grad.view(torch.int32))) == 0
    first = (rows - 3) * dim + 100
    part = torch.full((3 * dim - 200,), 5.0, device=DEV)
    layers.zero_embedding_grad(order, rows, d_out, part, ws, first=first, accumulate=True)
    full = torch.full((3 * dim,), 5.0, device=DEV)
    full[2 * dim:] += d_out[0].float() + d_out[11].float()
    assert torch.equal(part, full[100:3 * dim - 100])


def test_rows_far_apart():
    """Rows of every array with a stride of more than 2^31 elements."""
    n, dim = 3, 1000
    gen = generator(3)
    far, other = (torch.empty((n - 1) * FAR + dim, dtype=BF16, device=DEV) for _ in range(2))
    a, b = (torch.as_strided(t, (n, dim), (FAR, 1)) for t in (far, other))
    x = normal(gen, n, dim, dtype=BF16)
    a.copy_(x)
    mean, rstd = torch.empty(n, device=DEV), torch.empty(n, device=DEV)
    layers.zero_norm(a, b, mean, rstd)
    y = torch.empty_like(x)
    layers.zero_norm(x, y)
    assert torch.equal(b, y)
    d_y = normal(gen, n, dim, dtype=BF16)
    b.copy_(d_y)
    d_w, ws = torch.empty(dim, device=DEV), torch.empty(layers.zero_norm_grad_workspace_bytes(n, dim) // 4, device=DEV)
    layers.zero_norm_grad(b, a, mean, rstd, a, ws, d_weight=d_w)             # d_x over x
    d_x, d_w1 = torch.empty_like(x), torch.empty_like(d_w)
    layers.zero_norm_grad(d_y, x, mean, rstd, d_x, ws, d_weight=d_w1)
    assert torch.equal(a, d_x) and torch.equal(d_w, d_w1)
    tokens = torch.tensor([1, 0, 1], device=DEV)
    table = normal(gen, 2, dim, dtype=BF16)
    layers.zero_embedding(tokens, table, a)
    assert torch.equal(a, table[tokens])
    grad, grad1 = torch.empty(2, dim, device=DEV), torch.empty(2, dim, device=DEV)
    ws = torch.empty(layers.zero_embedding_grad_workspace_bytes(n, dim) // 4, device=DEV)
    layers.zero_embedding_grad(order_of(tokens, 2), 2, b, grad, ws)
    layers.zero_embedding_grad(order_of(tokens, 2), 2, d_y, grad1, ws)
    assert torch.equal(grad, grad1)


@pytest.mark.parametrize("dim,dtype", [(3, F32), (24, BF16), (300, BF16)])
def test_more_rows_than_a_launch(dim, dtype):
    """2^21 rows a launch of the norm: the rows behind are as those in front of it, bit by bit."""
    n, k = (1 << 21) + 1000, 1000
    gen = generator(dim)
    block = normal(gen, k, dim, dtype=dtype)
    x = torch.empty(n, dim, dtype=dtype, device=DEV)
    x[:k], x[k:n - k], x[n - k:] = block, 0.5, block
    res, total, y = x.clone(), torch.empty_like(x), torch.empty_like(x)
    mean, rstd = torch.full((n,), float("nan"), device=DEV), torch.full((n,), float("nan"), device=DEV)
    layers.zero_norm(x, y, mean, rstd, residual=res, total=total)
    for t in (y, total, mean, rstd):
        assert torch.equal(t[:k], t[n - k:])
    assert (total[k:n - k] == 1).all() and (mean[k:n - k] == 1).all() and not torch.isnan(rstd).any()
    want, bound = C.norm_bounds(total[:k], None, None, 1e-5, False, dtype)
    C.close(y[:k], want[0], bound[0], "y")
    # the column sums over all rows: those of the blocks, since a constant row's normalised values are zero
    d_y = torch.zeros_like(x)
    d_y[:k] = d_y[n - k:] = normal(gen, k, dim, dtype=dtype)
    d_y[k:n - k] = 1.0
    d_w = torch.empty(dim, device=DEV)
    ws = torch.empty(layers.zero_norm_grad_workspace_bytes(n, dim) // 4, device=DEV)
    layers.zero_norm_grad(d_y, total, mean, rstd, None, ws, d_weight=d_w)
    _, d_want, _ = O.norm_grad(C.np64(d_y[:k]), C.np64(total[:k]), C.np64(mean[:k]), C.np64(rstd[:k]))
    size = (abs(C.np64(d_y[:k]) * (C.np64(total[:k]) - C.np64(mean[:k])[:, None]) * C.np64(rstd[:k])[:, None])).sum(0)
    C.close(d_w, 2 * d_want, 2 * (128 + n / 64 + 3) * C.U * size, "d_weight")
