"""The token-table and norm calls as a training program uses them: with the
rank's accumulated step, on streams, in graphs, two at a time."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from fsdp_sharded_mixed_zero_amd import synth, zero  # noqa: E402
from fsdp_sharded_mixed_zero_amd import layers  # noqa: E402
from fsdp_sharded_mixed_zero_amd.rank import RankShard  # noqa: E402
import layer_cases as C  # noqa: E402
from devbits import u16  # noqa: E402
from layer_cases import DEV, U, generator, normal  # noqa: E402
from oracle import layers as O  # noqa: E402
from oracle import step as S  # noqa: E402
from oracle.layout import build_layout  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32

# a table of 101 rows, a norm's weight and bias, a matrix: cut by four ranks inside a row
DIM, ROWS, TOKENS, MICRO = 40, 101, 70, 3
SIZES = (ROWS * DIM, DIM, DIM, DIM * 30)


def workload(n_d, rank):
    return synth.Workload("tables", SIZES, n_d=n_d, rank=rank, align=16, grad_std=1e-2, max_norm=0.5, seed=3)


def micro_batch(mb):
    gen = generator(100 + mb)
    n = TOKENS - 11 * mb
    return (C.draw_tokens(n, ROWS, mb, dtype=torch.int32 if mb % 2 else torch.int64),
            normal(gen, n, DIM, std=1e-2, dtype=BF16 if mb != 1 else F32), 0.5 if mb == 2 else 1.0)


def run_rank(n_d, rank, dense, absent=()):
    wl = workload(n_d, rank)
    rs = RankShard(wl, accum_steps=MICRO, tables={0: {"dim": DIM, "tokens": TOKENS, "dense": dense}})
    kept = []

    def before_micro(mb):
        rs.fill_grads(50 + mb)
        kept.append([None if g is None else g.clone() for g in rs.grads])
        return {} if mb in absent else {0: micro_batch(mb)}

    master = torch.empty(rs.shard, device=DEV)
    m, v = torch.empty_like(master), torch.empty_like(master)
    zero.zero_state_export(rs.state, master, m, v, rs.shard)
    state = [t.cpu().numpy() for t in (master, m, v)]
    rs.step(7, before_micro=before_micro)
    torch.cuda.synchronize()
    return wl, rs, kept, state


@pytest.mark.parametrize("dense", [False, True])
@pytest.mark.parametrize("n_d,rank", [(1, 0), (4, 0), (4, 1), (4, 2), (4, 3)])
def test_accumulated_step_with_a_table(dense, n_d, rank):
    """The accumulator is the sum over the micro-batches of the packed dense
    gradients and the table's gradients; the step that follows is the oracle's on it."""
    wl, rs, kept, state = run_rank(n_d, rank, dense, absent=(1,) if rank == 2 else ())
    lay = build_layout(wl.sizes, n_d, rank, wl.align)
    lo, n = lay.shard_begin, lay.shard
    want, size = np.zeros(lay.padded), np.zeros(lay.padded)
    adds = np.zeros(lay.padded)
    for mb in range(MICRO):
        off = 0
        for i, g in enumerate(kept[mb]):
            if g is not None:
                g = C.np64(g)
                want[off:off + g.size] += g
                size[off:off + g.size] += np.abs(g)
                adds[off:off + g.size] += 1
            off += wl.sizes[i]
        if rank == 2 and mb == 1:
            continue
        tok, d, scale = micro_batch(mb)
        part, bound = C.embedding_grad_want(tok, d, ROWS, scale)
        want[:SIZES[0]] += part.ravel()
        size[:SIZES[0]] += np.abs(part).ravel() + bound.ravel() / U      # its own bound, in the units of size * u
        adds[:SIZES[0]] += 1
    acc = rs.acc.cpu().numpy().astype(np.float64)
    err, bound = np.abs(acc - want[lo:lo + n]), (adds * U * size)[lo:lo + n]
    assert (err <= C.SLACK * bound).all(), np.flatnonzero(err > C.SLACK * bound)[:5]
    assert (np.abs(want[lo:lo + n]) > 0).any()
    # the step reads the accumulator
    acc32 = rs.acc.cpu().numpy()
    own = S.sqnorm_f32(acc32)
    got = float(rs.rank_sq[rank])
    assert abs(np.sqrt(got) - np.sqrt(own)) <= 1e-6 * np.sqrt(own)
    coef = S.clip_coef(float(rs.rank_sq.sum()), wl.max_norm)
    hp = S.AdamWHParams(lr=wl.lr, beta1=wl.beta1, beta2=wl.beta2, eps=wl.eps, weight_decay=wl.weight_decay,
                        max_norm=wl.max_norm)
    _, _, _, param = S.adamw_step_f32grad(acc32, *state, 7, hp, coef)
    bits = u16(rs.param_shard).astype(np.int32)
    assert (np.abs(bits - param.astype(np.int32)) <= 1).all()
    # and the lookup reads what the step wrote, where the rank owns all of a row
    for i, s, d, k in rs.segments:
        if i == 0:
            first, last = -(-s // DIM), (s + k) // DIM
            tok = torch.arange(first, last, device=DEV)
            out = torch.empty(len(tok), DIM, dtype=BF16, device=DEV)
            layers.zero_embedding(tok, rs.params[0].view(ROWS, DIM), out)
            at = d + first * DIM - s
            assert torch.equal(out.flatten(), rs.param_shard[at:at + out.numel()])


def test_tables_that_do_not_fit_are_refused():
    wl = workload(1, 0)
    with pytest.raises(ValueError, match="accum_steps"):
        RankShard(wl, tables={0: {"dim": DIM, "tokens": 4}})
    with pytest.raises(ValueError, match="no table"):
        RankShard(wl, accum_steps=2, tables={0: {"dim": 7, "tokens": 4}})
    with pytest.raises(ValueError, match="no table"):
        RankShard(wl, accum_steps=2, tables={0: {"dim": 0, "tokens": 4}})
    with pytest.raises(ValueError, match="no table"):
        RankShard(wl, accum_steps=2, tables={9: {"dim": DIM, "tokens": 4}})
    rs = RankShard(wl, accum_steps=2, tables={0: {"dim": DIM, "tokens": 4}})
    five = (torch.zeros(5, dtype=torch.int32, device=DEV), torch.zeros(5, DIM, device=DEV))
    with pytest.raises(ValueError, match="5 tokens"):
        rs.step(1, before_micro=lambda mb: {0: five})
    with pytest.raises(ValueError, match="not among"):
        rs.step(1, before_micro=lambda mb: {1: five})


@pytest.mark.parametrize("tokens,shape", [(3, (4, DIM)), (4, (3, DIM)), (4, (4, DIM - 1)), (4, (2, 2 * DIM)), (4, (4 * DIM,))])
def test_a_table_gradient_of_another_shape_is_refused(tokens, shape):
    """Also where the rank's part would fit the other shape."""
    rs = RankShard(workload(4, 0), accum_steps=2, tables={0: {"dim": DIM, "tokens": 8}})
    given = (torch.zeros(tokens, dtype=torch.int32, device=DEV), torch.zeros(*shape, device=DEV))
    with pytest.raises(ValueError, match="rows of"):
        rs.step(1, before_micro=lambda mb: {0: given})


def test_bytes_of_a_step_leave_a_table_out():
    wl = workload(1, 0)
    without = RankShard(wl, accum_steps=MICRO).bytes_per_step()
    dense, by_tokens = (RankShard(wl, accum_steps=MICRO, tables={0: {"dim": DIM, "tokens": 4, "dense": d}}).bytes_per_step()
                        for d in (True, False))
    assert dense == without
    table = SIZES[0]
    assert by_tokens == {**without, "pack": without["pack"] - MICRO * 4 * table,
                         "accumulate": without["accumulate"] - (6 + 10 * (MICRO - 1)) * table}


class Pass:
    """One forward and backward pass: lookup, norm with the residual, and back. With the gradients of a loss that is
    the sum of y times a constant."""

    def __init__(self, n, rows, dim, seed, part=None):
        gen = generator(seed)
        self.n, self.rows, self.dim = n, rows, dim
        self.first, self.count = part or (0, rows * dim)
        self.table, self.weight, self.bias = normal(gen, rows, dim, dtype=BF16), normal(gen, dim), normal(gen, dim)
        self.residual, self.d_y, self.d_skip = (normal(gen, n, dim, dtype=BF16) for _ in range(3))
        self.tokens = C.draw_tokens(n, rows, seed)
        self.h, self.total, self.y, self.d_h = (torch.empty(n, dim, dtype=BF16, device=DEV) for _ in range(4))
        self.mean, self.rstd = torch.empty(n, device=DEV), torch.empty(n, device=DEV)
        self.acc = torch.zeros(self.count, device=DEV)
        self.d_w, self.d_b = torch.zeros(dim, device=DEV), torch.zeros(dim, device=DEV)
        self.order = torch.empty(layers.zero_token_order_bytes(n, rows) // 4, dtype=torch.int32, device=DEV)
        self.ws = torch.empty(max(layers.zero_embedding_grad_workspace_bytes(n, dim),
                                  layers.zero_norm_grad_workspace_bytes(n, dim)) // 4, device=DEV)

    def draw(self, seed):
        self.tokens.copy_(C.draw_tokens(self.n, self.rows, seed))
        self.d_y.copy_(normal(generator(seed), self.n, self.dim, dtype=BF16))

    def run(self, stream=None):
        kw = dict(stream=stream)
        layers.zero_embedding(self.tokens, self.table, self.h, scale=2.0, **kw)
        layers.zero_norm(self.h, self.y, self.mean, self.rstd, weight=self.weight, bias=self.bias,
                         residual=self.residual, total=self.total, **kw)
        layers.zero_norm_grad(self.d_y, self.total, self.mean, self.rstd, self.d_h, self.ws, weight=self.weight,
                              d_weight=self.d_w, d_bias=self.d_b, d_total=self.d_skip, accumulate=True, **kw)
        layers.zero_token_order(self.tokens, self.rows, self.order, **kw)
        layers.zero_embedding_grad(self.order, self.rows, self.d_h, self.acc, self.ws, scale=2.0, first=self.first,
                                   accumulate=True, **kw)

    def outputs(self):
        return [t.clone() for t in (self.h, self.total, self.y, self.mean, self.rstd, self.d_h, self.acc, self.d_w, self.d_b)]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def test_chain_against_differences():
    """The gradients of the chain in fp64 by differences of the oracle's forward pass, at sampled table and weight
    entries. The chain rounds the lookup, the sum and the gradient of the rows to bf16 (2^-8 each, relative to a value),
    so a gradient entry may be off by 4 * 2^-8 of the sum of the magnitudes that enter it; differences with step
    1e-4 add less than that."""
    p = Pass(50, 20, 48, 5)
    p.d_skip.zero_()
    p.run()
    tok, W, w, b = p.tokens.cpu().numpy(), C.np64(p.table), C.np64(p.weight), C.np64(p.bias)
    res, dy = C.np64(p.residual), C.np64(p.d_y)

    def loss(W, w, b):
        s = O.embedding(tok, W, 2.0) + res
        return (O.norm(s, w, b)[0] * dy).sum()

    r = np.random.default_rng(0)
    grads = [C.np64(p.acc).reshape(20, 48), C.np64(p.d_w), C.np64(p.d_b)]
    s = O.embedding(tok, W, 2.0) + res
    _, _, rstd = O.norm(s, w, b)
    for arg, g in zip((0, 1, 2), grads):
        for _ in range(12):
            at = tuple(r.integers(0, k) for k in g.shape)
            vals = []
            for sign in (1, -1):
                a = [W.copy(), w.copy(), b.copy()]
                a[arg][at] += sign * 1e-4
                vals.append(loss(*a))
            want = (vals[0] - vals[1]) / 2e-4
            if arg == 0:
                rows = np.flatnonzero(tok == at[0])
                # |d_x| <= rstd (|g| + mean|g| + |xh| mean|g xh|), with |xh| below 5 and means below the largest |g|
                size = 2.0 * sum(rstd[t] * 27 * np.abs(dy[t] * w).max() for t in rows)
            else:
                size = (np.abs(dy) * 5)[:, at[0]].sum()
            assert abs(g[at] - want) <= 4 * 2.0 ** -8 * size + 1e-6, (arg, at, g[at], want)


@pytest.mark.parametrize("n,rows,dim", [(60, 30, 40), (5000, 300, 264), (13000, 700, 72)])
def test_chain_on_another_stream_and_twice_at_once(n, rows, dim):
    """On a stream that is not the current one, and two chains at a time, the results are those of one after the other."""
    a, b = Pass(n, rows, dim, 1), Pass(n, rows, dim, 2, part=(dim // 2, (rows - 3) * dim + 1))
    a.run(), b.run()
    torch.cuda.synchronize()
    want = a.outputs(), b.outputs()
    for p in (a, b):
        p.acc.zero_(), p.d_w.zero_(), p.d_b.zero_()
        for t in (p.h, p.total, p.y, p.mean, p.rstd, p.d_h):
            t.fill_(float("nan"))
    torch.cuda.synchronize()
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    a.run(one), b.run(two)
    torch.cuda.synchronize()
    assert same(a.outputs(), want[0]) and same(b.outputs(), want[1])


@pytest.mark.parametrize("n,rows,dim", [(60, 30, 40), (5000, 300, 264), (13000, 700, 72), (40, 20, 17000)])
def test_chain_in_a_graph(n, rows, dim):
    """Captured once, replayed several times on new tokens and gradients with eager work between: the same bits as
    eager calls on the same inputs. The workspace is the graph's and the eager calls' alike."""
    graphed, eager = Pass(n, rows, dim, 1), Pass(n, rows, dim, 1)
    graphed.run()                                # warm-up
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        graphed.run()
    for p in (graphed, eager):
        p.acc.zero_(), p.d_w.zero_(), p.d_b.zero_()
    for rep in range(4):
        graphed.draw(20 + rep), eager.draw(20 + rep)
        eager.run()
        graph.replay()
        torch.cuda.synchronize()
        assert same(graphed.outputs(), eager.outputs()), rep


def test_a_gradient_is_the_same_every_time():
    p = Pass(9000, 400, 520, 9)
    p.run()
    want = p.outputs()
    for _ in range(3):
        p.acc.zero_(), p.d_w.zero_(), p.d_b.zero_()
        p.run()
        assert same(p.outputs(), want)


def test_two_parts_from_one_order():
    """One order, the table's gradient in three parts and whole: the same bits."""
    p = Pass(900, 50, 100, 4)
    p.run()
    whole = torch.empty(50 * 100, device=DEV)
    layers.zero_embedding_grad(p.order, 50, p.d_h, whole, p.ws)
    cuts = [0, 1234, 1235, 5000]
    for lo, hi in zip(cuts, cuts[1:]):
        part = torch.empty(hi - lo, device=DEV)
        layers.zero_embedding_grad(p.order, 50, p.d_h, part, p.ws, first=lo)
        assert torch.equal(part, whole[lo:hi])


def test_a_buffer_for_the_largest_batch_serves_all():
    n, rows, dim = 5000, 64, 24
    order = torch.empty(layers.zero_token_order_bytes(n, rows) // 4, dtype=torch.int32, device=DEV)
    ws = torch.empty(layers.zero_embedding_grad_workspace_bytes(n, dim) // 4, device=DEV)
    for k in (4096, 4097, 1, 0, 5000):
        tokens, d = C.draw_tokens(k, rows, k), normal(generator(k), k, dim)
        grad = torch.empty(rows, dim, device=DEV)
        layers.zero_token_order(tokens, rows, order)
        layers.zero_embedding_grad(order, rows, d, grad, ws)
        want, bound = C.embedding_grad_want(tokens, d, rows, 1.0)
        C.close(grad, want, C.stored(bound, want, F32), str(k))
