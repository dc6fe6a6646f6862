"""Token tables and norms on the GPU against the fp64 oracle, at the sizes, types,
strides and tokens where they can go wrong. The tolerances are derived in layer_cases.py."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from fsdp_sharded_mixed_zero_amd import layers

import layer_cases as C  # noqa: E402
from layer_cases import DEV, U, close, generator, half_step, normal, stored  # noqa: E402
from oracle import layers as O  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32


# ------------------------------------------------------------------ lookup

@pytest.mark.parametrize("n,rows,dim", [(1, 1, 1), (3, 7, 5), (5, 100, 8), (67, 33, 129), (130, 1009, 777), (9, 50, 2049)])
@pytest.mark.parametrize("table_type,out_type", [(BF16, BF16), (BF16, F32), (F32, BF16), (F32, F32)])
@pytest.mark.parametrize("ids", [torch.int32, torch.int64])
def test_embedding(n, rows, dim, table_type, out_type, ids):
    gen = generator(n + dim)
    table = normal(gen, rows, dim, dtype=table_type)
    tokens = C.draw_tokens(n, rows, n, dtype=ids)
    out, whole = C.rows_of(torch.zeros(n, dim, dtype=out_type, device=DEV), dim + 3)
    layers.zero_embedding(tokens, table, out, scale=1.5)
    want = O.embedding(tokens.cpu().numpy(), C.np64(table), 1.5)
    close(out, want, (U + half_step(out_type) * (1 + U)) * np.abs(want), "out")
    assert torch.isnan(whole[:, dim:]).all()
    assert (C.np64(out)[want == 0] == 0).all()


@pytest.mark.parametrize("by", [1, 3, 7])
def test_embedding_at_odd_addresses(by):
    gen = generator(by)
    table = C.shifted(normal(gen, 60, 72, dtype=BF16), by)
    tokens = C.draw_tokens(50, 60, by)
    out = C.shifted(torch.zeros(50, 72, dtype=BF16, device=DEV), by)
    layers.zero_embedding(tokens, table, out)
    assert np.array_equal(C.np64(out), O.embedding(tokens.cpu().numpy(), C.np64(table)))


def test_embedding_of_no_tokens():
    out = torch.zeros(0, 8, dtype=BF16, device=DEV)
    layers.zero_embedding(torch.zeros(0, dtype=torch.int64, device=DEV), normal(generator(0), 4, 8, dtype=BF16), out)
    layers.zero_embedding(torch.zeros(0, 3, dtype=torch.int32, device=DEV), normal(generator(0), 4, 8, dtype=F32), out)


# ------------------------------------------------------------------- sort

def order_of(tokens, rows):
    order = torch.full((layers.zero_token_order_bytes(tokens.numel(), rows) // 4,), -7, dtype=torch.int32, device=DEV)
    layers.zero_token_order(tokens, rows, order)
    return order


@pytest.mark.parametrize("n", [0, 1, 2, 31, 32, 33, 65, 1000, 4099, 8191, 8192, 8193, 10000, 20000])
@pytest.mark.parametrize("rows", [1, 2, 31, 512, 50257, 300000])
@pytest.mark.parametrize("kind", ["mixed", "same", "distinct", "none"])
def test_token_order(n, rows, kind):
    """The gradient of one column of ones and of positions shows the order only as sums, so the
    order's first parts are read here: the rows and the positions."""
    ids = torch.int32 if (n + rows) % 2 else torch.int64
    tokens = C.draw_tokens(n, rows, n + rows, kind, ids)
    order = order_of(tokens, rows).cpu().numpy()
    row, pos = O.token_order(tokens.cpu().numpy(), rows)
    up = (n + 7) // 8 * 8 + 8
    assert order[:len(row)].tolist() == row
    assert order[up:up + len(row)].tolist() == pos
    assert (order[len(row):n] == rows).all()


@pytest.mark.parametrize("n", [4096, 4097, 5001, 8191, 8192, 8193, 12289, 16383, 16384, 16385])
@pytest.mark.parametrize("rows", [1, 2, 255, 256, 257, 4000, 50257, 131071, 131072])
def test_token_order_of_some_thousand(n, rows):
    """Tokens spread over the table, outside it, in few of its consecutive rows, all on its last row, and in order."""
    gen = generator(n + rows)
    pick = lambda lo, hi: torch.randint(lo, hi, (n,), generator=gen, device=gen.device).to(DEV)  # noqa: E731
    few = max(0, rows // 2 - 70)
    lists = [pick(-rows // 3 - 1, rows + rows // 3 + 2), pick(few, min(rows, few + 140)), torch.full((n,), rows - 1, device=DEV),
             torch.where(pick(0, 2) == 0, pick(0, rows), pick(0, 1) + rows // 3), pick(0, rows).sort().values]
    lists[0][n // 2] = 2 ** 32 + rows // 2       # outside the table, whatever its lower half says
    lists[0][n // 3] = -2 ** 32 + rows // 2
    for k, tokens in enumerate(lists):
        for t in (tokens, tokens.to(torch.int32)) if k else (tokens,):
            order = order_of(t, rows).cpu().numpy()
            row, pos = O.token_order(t.cpu().numpy(), rows)
            up = (n + 7) // 8 * 8 + 8
            assert order[:len(row)].tolist() == list(row) and order[up:up + len(row)].tolist() == list(pos), k
            assert (order[len(row):n] == rows).all()


def test_token_order_of_a_wide_table():
    """Three passes of the sort."""
    rows, n = 16_000_001, 9500
    tokens = C.draw_tokens(n, rows, 5)
    for t in (tokens, tokens[:3000].clone()):
        order = order_of(t, rows).cpu().numpy()
        row, pos = O.token_order(t.cpu().numpy(), rows)
        up = (len(t) + 7) // 8 * 8 + 8
        assert order[:len(row)].tolist() == row and order[up:up + len(row)].tolist() == pos


# -------------------------------------------------------- table's gradient

def table_grad(tokens, rows, d_out, grad, **kw):
    n, dim = d_out.shape
    ws = torch.full((layers.zero_embedding_grad_workspace_bytes(n, dim) // 4,), float("nan"), device=DEV)
    layers.zero_embedding_grad(order_of(tokens, rows), rows, d_out, grad, ws, **kw)


@pytest.mark.parametrize("n,rows,dim", [(1, 1, 1), (2, 3, 5), (40, 7, 8), (33, 50, 300), (100, 2, 64), (700, 90, 513),
                                        (4500, 61, 40), (5000, 6000, 12)])
@pytest.mark.parametrize("out_type,grad_type", [(BF16, BF16), (BF16, F32), (F32, BF16), (F32, F32)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_embedding_grad(n, rows, dim, out_type, grad_type, accumulate):
    for kind in ("mixed", "same", "distinct", "none"):
        gen = generator(n + dim)
        tokens = C.draw_tokens(n, rows, n, kind)
        d_out, _ = C.rows_of(normal(gen, n, dim, dtype=out_type), dim + 5)
        if kind == "mixed":        # rows of tokens outside the table are not read
            outside = (tokens < 0) | (tokens >= rows)
            d_out[outside] = float("nan")
        old = normal(gen, rows, dim, dtype=grad_type)
        grad = old.clone() if accumulate else torch.full_like(old, float("nan"))
        table_grad(tokens, rows, d_out, grad, scale=0.75, accumulate=accumulate)
        want, bound = C.embedding_grad_want(tokens, torch.nan_to_num(d_out), rows, 0.75, old if accumulate else None)
        close(grad, want, stored(bound, want, grad_type), kind)
        if accumulate:             # rows without a token keep their bits
            met = torch.zeros(rows, dtype=torch.bool, device=DEV)
            met[tokens[(tokens >= 0) & (tokens < rows)].long()] = True
            assert torch.equal(grad[~met], old[~met])


@pytest.mark.parametrize("first,count", [(0, 0), (0, 1), (1, 1), (7, 30), (0, 37 * 5), (37 * 5, 37), (37 * 3 + 11, 37 * 9),
                                         (37 * 20 + 36, 2), (37 * 39 + 1, 36), (5, 37 * 40 - 5)])
@pytest.mark.parametrize("out_type,grad_type", [(BF16, BF16), (BF16, F32), (F32, F32)])
def test_embedding_grad_of_a_part(first, count, out_type, grad_type):
    """Parts that begin and end inside rows; what lies beside the part keeps its bits."""
    rows, dim, n = 40, 37, 500
    gen = generator(first + count)
    tokens = C.draw_tokens(n, rows, first)
    d_out = normal(gen, n, dim, dtype=out_type)
    whole = torch.full((rows * dim,), float("nan"), dtype=grad_type, device=DEV)
    table_grad(tokens, rows, d_out, whole)
    old = normal(gen, rows * dim, dtype=grad_type)
    added = old.clone()
    table_grad(tokens, rows, d_out, added, accumulate=True)
    for accumulate in (False, True):
        buf = normal(gen, count + 20, dtype=grad_type)
        keep = buf.clone()
        if accumulate:
            buf[9:9 + count] = old[first:first + count]
        table_grad(tokens, rows, d_out, buf[9:9 + count], first=first, accumulate=accumulate)
        assert torch.equal(buf[:9], keep[:9]) and torch.equal(buf[9 + count:], keep[9 + count:])
        assert torch.equal(buf[9:9 + count], (added if accumulate else whole)[first:first + count])


def test_embedding_grad_of_long_runs():
    """Half of 40000 tokens on one row, as a batch padded with a real token has them."""
    n, rows, dim = 40000, 300, 24
    gen = generator(1)
    tokens = C.draw_tokens(n, rows, 2)
    tokens[::2] = 17
    d_out = normal(gen, n, dim, dtype=BF16)
    grad = torch.empty(rows, dim, device=DEV)
    table_grad(tokens, rows, d_out, grad)
    want, bound = C.embedding_grad_want(tokens, d_out, rows, 1.0)
    close(grad, want, stored(bound, want, F32), "grad")
    again = torch.empty_like(grad)
    table_grad(tokens, rows, d_out, again)
    assert torch.equal(grad, again)


@pytest.mark.parametrize("runs", [[64] * 9, [63, 65, 64, 128, 1, 7, 500], [128, 256, 3, 125, 1000], [1, 127, 128, 384, 9], [2000],
                                  [17, 4096, 15], [5, 20000, 200, 128, 1], [128] * 40, [8192 + 128 * 3 - 1, 1, 4000], [120, 5000, 8]])
@pytest.mark.parametrize("dim", [5, 300, 1100])
def test_embedding_grad_of_runs_at_the_pieces_borders(runs, dim):
    """Runs that begin and end on, before and behind the borders of pieces and of groups of them, with whole numbers:
    every sum is exact, in any order."""
    rows = len(runs)
    r = np.random.default_rng(sum(runs) + dim)
    tokens = np.repeat(np.arange(rows), runs)
    at = r.permutation(len(tokens))
    d = r.integers(-4, 5, (len(tokens), dim)).astype(np.float32)
    want = np.stack([d[tokens == k].sum(0) for k in range(rows)])
    shuffled = torch.from_numpy(tokens[at]).to(DEV)
    for grad_type in (F32, BF16):
        d_out = torch.from_numpy(d[at]).to(DEV).to(BF16 if grad_type == F32 else F32)
        grad = torch.full((rows, dim), 2.0, dtype=grad_type, device=DEV)
        table_grad(shuffled, rows, d_out, grad)
        exact = torch.from_numpy(want).to(DEV)
        assert torch.equal(grad, exact.to(grad_type))
        table_grad(shuffled, rows, d_out, grad, accumulate=True)
        assert torch.equal(grad, (exact.to(grad_type).float() + exact).to(grad_type))


def test_embedding_grad_keeps_infinities_and_nans_to_their_elements():
    n, rows, dim = 90, 12, 20
    tokens = C.draw_tokens(n, rows, 3, "distinct")
    d_out = normal(generator(3), n, dim)
    d_out[5, 3], d_out[40, 7], d_out[41, 8] = float("nan"), float("inf"), -float("inf")
    grad = torch.empty(rows, dim, device=DEV)
    table_grad(tokens, rows, d_out, grad)
    bad = torch.zeros(rows, dim, dtype=torch.bool, device=DEV)
    bad[tokens[5], 3] = bad[tokens[40], 7] = bad[tokens[41], 8] = True
    assert torch.equal(~torch.isfinite(grad), bad)


# -------------------------------------------------------------------- norm

SHAPES = [(1, 1), (3, 2), (2, 7), (5, 64), (17, 100), (9, 129), (6, 512), (5, 777), (4, 1024), (3, 1600), (4, 2944),
          (3, 4099), (2, 8192), (2, 12001), (2, 16385), (1, 20000), (2, 33000), (1025, 1301), (1100, 700)]


def norm_case(n, dim, dtype, w_type, seed, offset=0.3):
    gen = generator(seed)
    x = normal(gen, n, dim, dtype=F32)
    x = (x * (normal(gen, dim) * 0.5).exp() + offset).to(dtype)
    return gen, x, normal(gen, dim, dtype=w_type), normal(gen, dim, dtype=w_type)


@pytest.mark.parametrize("n,dim", SHAPES)
@pytest.mark.parametrize("dtype,w_type", [(BF16, BF16), (BF16, F32), (F32, BF16), (F32, F32)])
@pytest.mark.parametrize("rms", [False, True])
def test_norm(n, dim, dtype, w_type, rms):
    for residual in (False, True):
        gen, x, w, b = norm_case(n, dim, dtype, w_type, n * dim)
        x, _ = C.rows_of(x, dim + 3)
        y, y_whole = C.rows_of(torch.zeros(n, dim, dtype=dtype, device=DEV), dim + 1)
        mean, rstd = torch.empty(n, device=DEV), torch.empty(n, device=DEV)
        res = normal(gen, n, dim, dtype=dtype) if residual else None
        total = torch.empty(n, dim, dtype=dtype, device=DEV) if residual else None
        layers.zero_norm(x, y, mean, rstd, weight=w, bias=b, eps=1e-5, residual=res, total=total, rms=rms)
        s = x
        if residual:
            want = C.np64(x) + C.np64(res)
            close(total, want, (U + half_step(dtype) * (1 + U)) * np.abs(want), "total")
            s = total
        want, bound = C.norm_bounds(s, w, b, 1e-5, rms, dtype)
        for got, v, e, what in zip((y, mean, rstd), want, bound, ("y", "mean", "rstd")):
            close(got, v, e, f"{what}, residual {residual}")
        assert torch.isnan(y_whole[:, dim:]).all()


@pytest.mark.parametrize("dim", [24, 700, 5000, 40000])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_norm_of_far_means_and_without_vectors(dim, dtype):
    """A mean 100 times the deviation, no weight, no bias, no statistics asked for; in place."""
    gen, x, _, _ = norm_case(5, dim, dtype, F32, dim, offset=100.0)
    want, bound = C.norm_bounds(x, None, None, 1e-5, False, dtype)
    layers.zero_norm(x, x)
    close(x, want[0], bound[0], "y")


def test_norm_in_place_with_residual():
    for dim in (40, 3000, 17000):
        gen, x, w, b = norm_case(4, dim, BF16, BF16, dim)
        res = normal(gen, 4, dim, dtype=BF16)
        y, total = torch.empty_like(x), torch.empty_like(x)
        layers.zero_norm(x, y, weight=w, bias=b, residual=res, total=total)
        y2, res2 = torch.empty_like(x), res.clone()
        layers.zero_norm(x, y2, weight=w, bias=b, residual=res2, total=res2)      # the stream of residuals, updated
        assert torch.equal(y, y2) and torch.equal(total, res2)
        x2 = x.clone()
        layers.zero_norm(x2, x2, weight=w, bias=b, residual=res, total=total)     # y over x
        assert torch.equal(y, x2)


def test_norm_of_constant_rows_and_bad_values():
    """A row without deviation gives the bias; a NaN or an infinity spoils its own row only."""
    x = normal(generator(4), 6, 96)
    x[1] = 3.25
    x[2, 5] = float("nan")
    x[3, 6] = float("inf")
    y, mean, rstd = torch.empty_like(x), torch.empty(6, device=DEV), torch.empty(6, device=DEV)
    b = normal(generator(5), 96)
    layers.zero_norm(x, y, mean, rstd, bias=b)
    assert torch.equal(y[1], b) and mean[1] == 3.25
    assert not torch.isfinite(y[2]).any() and not torch.isfinite(y[3, 6])
    ok = [0, 1, 4, 5]
    want, bound = C.norm_bounds(x[ok], None, b, 1e-5, False, F32)
    close(y[ok], want[0], bound[0], "y")


def test_norm_of_no_rows():
    x = torch.zeros(0, 16, device=DEV)
    layers.zero_norm(x, torch.empty_like(x), torch.zeros(0, device=DEV), torch.zeros(0, device=DEV))


# --------------------------------------------------------- norm's gradient

def workspace(n, dim):
    return torch.full((layers.zero_norm_grad_workspace_bytes(n, dim) // 4,), float("nan"), device=DEV)


@pytest.mark.parametrize("n,dim", SHAPES + [(700, 33), (300, 257), (600, 4099), (40, 17000)])
@pytest.mark.parametrize("dtype,w_type,g_type", [(BF16, BF16, F32), (BF16, F32, BF16), (F32, BF16, BF16), (F32, F32, F32)])
@pytest.mark.parametrize("rms", [False, True])
def test_norm_grad(n, dim, dtype, w_type, g_type, rms):
    for accumulate, skip in ((False, True), (True, False)):
        gen, x, w, _ = norm_case(n, dim, dtype, w_type, n + dim)
        x, _ = C.rows_of(x, dim + 3)
        d_y, _ = C.rows_of(normal(gen, n, dim, dtype=dtype), dim + 9)
        d_total = normal(gen, n, dim, dtype=dtype) if skip else None
        _, mean, rstd = (torch.from_numpy(v).float().to(DEV) for v in O.norm(C.np64(x), rms=rms))
        d_x, whole = C.rows_of(torch.zeros(n, dim, dtype=dtype, device=DEV), dim + 1)
        old = normal(gen, 2, dim, dtype=g_type)
        d_w, d_b = old.clone() if accumulate else torch.full_like(old, float("nan"))
        layers.zero_norm_grad(d_y, x, mean, rstd, d_x, workspace(n, dim), weight=w, d_weight=d_w, d_bias=d_b,
                              d_total=d_total, accumulate=accumulate, rms=rms)
        want, bound = C.norm_grad_want(d_y, x, mean, rstd, w, d_total, rms, dtype)
        close(d_x, want[0], bound[0], "d_x")
        for got, v, e, before, what in zip((d_w, d_b), want[1:], bound[1:], C.np64(old), ("d_weight", "d_bias")):
            if accumulate:
                v, e = v + before, e + U * np.abs(v + before)
            close(got, v, stored(e, v, g_type), what)
        assert torch.isnan(whole[:, dim:]).all()


@pytest.mark.parametrize("dim", [1, 3, 7, 8, 20, 100, 200, 400, 777, 1100, 1600, 2100, 2944, 3500, 4096, 4097, 5500, 8192])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_norm_grad_at_the_row_counts_where_kernels_change(dim, dtype):
    """The last number of rows that one launch takes, the next one, and d_x over x there."""
    last = 512 if dim > 4096 else 256
    for n in (last, last + 1):
        gen, x, w, _ = norm_case(n, dim, dtype, dtype, n + dim)
        d_y, d_total = normal(gen, n, dim, dtype=dtype), normal(gen, n, dim, dtype=dtype)
        _, mean, rstd = (torch.from_numpy(v).float().to(DEV) for v in O.norm(C.np64(x)))
        d_x, d_w, d_b = torch.empty_like(x), torch.empty(dim, device=DEV), torch.empty(dim, device=DEV)
        layers.zero_norm_grad(d_y, x, mean, rstd, d_x, workspace(n, dim), weight=w, d_weight=d_w, d_bias=d_b,
                              d_total=d_total)
        want, bound = C.norm_grad_want(d_y, x, mean, rstd, w, d_total, False, dtype)
        close(d_x, want[0], bound[0], "d_x")
        for got, v, e, what in zip((d_w, d_b), want[1:], bound[1:], ("d_weight", "d_bias")):
            close(got, v, stored(e, v, F32), what)
        one = torch.empty_like(d_w)
        layers.zero_norm_grad(d_y, x, mean, rstd, x, workspace(n, dim), weight=w, d_weight=one, d_total=d_total)
        assert torch.equal(x, d_x) and torch.equal(one, d_w)


@pytest.mark.parametrize("dim", [50, 1000, 6000, 18000])
def test_norm_grad_in_part_and_in_place(dim):
    """One output at a time, and d_x over each of its inputs, give the same bits."""
    n = 70
    gen, x, w, _ = norm_case(n, dim, BF16, BF16, dim)
    d_y, d_total = normal(gen, n, dim, dtype=BF16), normal(gen, n, dim, dtype=BF16)
    _, mean, rstd = (torch.from_numpy(v).float().to(DEV) for v in O.norm(C.np64(x)))
    d_x, (d_w, d_b) = torch.empty_like(x), torch.empty(2, dim, device=DEV)
    ws = workspace(n, dim)
    layers.zero_norm_grad(d_y, x, mean, rstd, d_x, ws, weight=w, d_weight=d_w, d_bias=d_b, d_total=d_total)
    one = torch.empty_like(d_w)
    layers.zero_norm_grad(d_y, x, mean, rstd, None, workspace(n, dim), d_weight=one, weight=w)
    assert torch.equal(one, d_w)
    layers.zero_norm_grad(d_y, x, mean, rstd, None, workspace(n, dim), d_bias=one)
    assert torch.equal(one, d_b)
    alone = torch.empty_like(x)
    layers.zero_norm_grad(d_y, x, mean, rstd, alone, weight=w, d_total=d_total)
    assert torch.equal(alone, d_x)
    for k in range(3):
        a = [d_y.clone(), x.clone(), d_total.clone()]
        layers.zero_norm_grad(a[0], a[1], mean, rstd, a[k], workspace(n, dim), weight=w, d_weight=one, d_total=a[2])
        assert torch.equal(a[k], d_x) and torch.equal(one, d_w)


def test_norm_grad_of_a_broadcast_gradient_and_without_weight():
    """d_y as one row for all (stride 0), as the gradient of a mean over rows arrives."""
    n, dim = 130, 600
    gen, x, _, _ = norm_case(n, dim, F32, F32, 8)
    d_y = normal(gen, 1, dim).expand(n, dim)
    _, mean, rstd = (torch.from_numpy(v).float().to(DEV) for v in O.norm(C.np64(x)))
    d_x, (d_w, d_b) = torch.empty_like(x), torch.empty(2, dim, device=DEV)
    layers.zero_norm_grad(d_y, x, mean, rstd, d_x, workspace(n, dim), d_weight=d_w, d_bias=d_b)
    want, bound = C.norm_grad_want(d_y, x, mean, rstd, None, None, False, F32)
    for got, v, e, what in zip((d_x, d_w, d_b), want, bound, ("d_x", "d_weight", "d_bias")):
        close(got, v, stored(e, v, F32), what)


@pytest.mark.parametrize("accumulate", [False, True])
def test_norm_grad_of_no_rows(accumulate):
    for dim in (40, 20000):
        x = torch.zeros(0, dim, device=DEV)
        d_w = torch.full((dim,), 2.0, device=DEV)
        empty = torch.zeros(0, device=DEV)
        layers.zero_norm_grad(x, x, empty, empty, torch.empty_like(x), workspace(0, dim), d_weight=d_w, accumulate=accumulate)
        assert (d_w == (2.0 if accumulate else 0.0)).all()
