"""The tensor-list calls as a rank's step uses them (TensorRank): against the
step over three state arrays and the oracle over several steps, a checkpoint
taken through fp32 moments, replayed from a graph, on several streams and from
several threads at once, with tensors beyond 2^31 elements and gradients
farther apart than 32-bit offsets reach."""

import threading

import numpy as np
import pytest

from fsdp_sharded_mixed_zero_amd import synth, tensors, zero
from fsdp_sharded_mixed_zero_amd.rank import RankShard, TensorRank
from oracle import state8 as S8
from oracle import step as O
from devbits import hp_of, u16
from tensor_lists import Case
from tolerance import ordered_f32
from test_gpu_tensors import check_codes, check32, check8, run_step, untouched

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda"

# a small model whose shard cuts through tensors, with odd sizes and padding at its end
ODD = synth.Workload("odd", tuple([5000, 33, 1, 70001, 257, 4096, 12345, 999]), n_d=3, rank=1, m_std=1e-4, v_std=1e-8,
                     step=7)
LAST = synth.Workload("last", ODD.sizes, n_d=3, rank=2, align=4096, m_std=1e-4, v_std=1e-8, step=7)


@pytest.mark.parametrize("wl", [synth.WORKLOADS["tiny"], ODD, LAST, synth.WORKLOADS["gpt2-1.5b"]], ids=lambda w: w.name)
def test_step32_is_the_state_array_step(wl):
    """Same inputs, same update. The two sums of squares differ in order, so
    the coefficients may differ by some 2^-52: equal in fp32, and a master
    recomputed in fp64 may round to the neighbour."""
    a, b = RankShard(wl, state_arrays=True), TensorRank(wl)
    for t in range(wl.step, wl.step + 3):
        a.step(t)
        b.step(t)
    torch.cuda.synchronize()
    ga, gb = float(a.rank_sq.sum()), float(b.rank_sq.sum())
    assert abs(ga - gb) <= 1e-12 * ga
    if np.float32(O.clip_coef(ga, wl.max_norm)) != np.float32(O.clip_coef(gb, wl.max_norm)):
        pytest.skip("the coefficients fall on two sides of an fp32 border")
    for k in ("master", "m", "v"):
        x, y = (getattr(r, k)[:a.real].cpu().numpy() for r in (a, b))
        assert np.abs(ordered_f32(x) - ordered_f32(y)).max() <= 1, k
    for i in a.touched:
        x, y = u16(a.params[i]).astype(np.int32), u16(b.params[i]).astype(np.int32)
        assert np.abs(x - y).max() <= 1, i
        outside = x == synth.SENTINEL
        assert np.array_equal(outside, y == synth.SENTINEL)


@pytest.mark.parametrize("wl", [synth.WORKLOADS["tiny"], ODD, LAST], ids=lambda w: w.name)
def test_step8_against_the_oracle_over_steps(wl):
    """Five steps with fresh gradients: every byte and scale of the moments as
    the oracle's chain of fp64 updates has them, masters within the bound of
    one step times the steps taken."""
    b = TensorRank(wl, state_bits=8)
    segs = b.segments
    cuts = np.cumsum([0] + [tensors.state8_blocks(n) for _, _, _, n in segs])

    def state():
        m, ms, v, vs = (x.view(torch.uint8).cpu().numpy() if x.dtype == torch.float8_e4m3fn else x.cpu().numpy()
                        for x in (b.m8, b.m_scale, b.v8, b.v_scale))
        return [(m[d:d + n], ms[cuts[k]:cuts[k + 1]], v[d:d + n], vs[cuts[k]:cuts[k + 1]])
                for k, (_, _, d, n) in enumerate(segs)]

    want = state()
    master = [b.master[d:d + n].cpu().numpy().astype(np.float64) for _, _, d, n in segs]
    bound = [np.zeros(n) for _, _, _, n in segs]
    ohp = O.AdamWHParams(lr=wl.lr, weight_decay=wl.weight_decay, max_norm=wl.max_norm)
    for t in range(wl.step, wl.step + 5):
        b.fill_grads(t)
        b.step(t)
        coef = O.clip_coef(O.global_sqnorm(b.rank_sq.cpu().numpy()), wl.max_norm)
        got = state()
        for k, (i, s, d, n) in enumerate(segs):
            g = (u16(b.grads[i])[s:s + n].astype(np.uint32) << 16).view(np.float32)
            old = master[k]
            master[k], m1, v1, want[k] = S8.adamw8_step(g, old, *want[k], t, ohp, coef)
            bound[k] += S8.update_bound(old, m1, v1, t, ohp)
            check_codes(got[k], want[k], f"step {t} segment {k}")
            # the bytes of a block whose scale differs by a step are as good; go on from the device's own
            want[k] = got[k]
            assert (np.abs(b.master[d:d + n].cpu().numpy() - master[k]) <= bound[k]).all(), (t, k)
            assert torch.equal(b.params[i][s:s + n], b.master[d:d + n].to(torch.bfloat16))
    for i in b.touched:      # nothing outside the rank's parts was written
        bits = u16(b.params[i])
        own = np.zeros(bits.size, bool)
        for j, s, _, n in segs:
            if j == i:
                own[s:s + n] = True
        assert (bits[~own] == synth.SENTINEL).all()


def test_groups_of_a_rank():
    """Norms and biases (one-dimensional tensors) in a group without decay."""
    wl = ODD
    base = dict(lr=wl.lr, beta1=wl.beta1, beta2=wl.beta2, eps=wl.eps, max_norm=wl.max_norm)
    small = lambda i: 1 if wl.sizes[i] < 5000 else 0  # noqa: E731
    r = TensorRank(wl, groups=[dict(base, weight_decay=0.5), dict(base, weight_decay=0.0)], group_of=small)
    before = r.master.clone()
    for i in r.touched:
        r.grads[i].zero_()
    r.m.zero_()
    r.step(wl.step)
    for i, _, d, n in r.segments:
        x = before[d:d + n]
        decayed = torch.addcmul(x, x, torch.tensor(-np.float32(wl.lr * 0.5), device=DEV)) if not small(i) else x
        assert (r.master[d:d + n] - decayed).abs().max() <= 2.0 ** -24 * x.abs().max()
        assert small(i) == 0 or torch.equal(r.master[d:d + n], x)


def test_checkpoint_through_fp32_moments():
    """Export, a new rank, import: the bytes come back, the scales within
    three roundings, and the next step goes on."""
    wl = ODD
    a, b = TensorRank(wl, state_bits=8), TensorRank(wl, state_bits=8, fill=False)
    a.step(wl.step)
    m, v = ([torch.empty(n, device=DEV) for _, _, _, n in a.segments] for _ in range(2))
    tensors.zero_tensors_state_export(a.list, m, v)
    tensors.zero_tensors_state_import(b.list, m, v)
    for k in ("m8", "v8"):
        assert torch.equal(getattr(a, k).view(torch.uint8), getattr(b, k).view(torch.uint8)), k
    for k in ("m_scale", "v_scale"):
        x, y = getattr(a, k), getattr(b, k)
        assert ((x - y).abs() <= 3 * 2.0 ** -24 * x).all(), k


@pytest.mark.parametrize("bits", [32, 8])
def test_graph_replays_equal_eager_steps(bits):
    wl = synth.WORKLOADS["tiny"]
    eager, graphed = TensorRank(wl, state_bits=bits), TensorRank(wl, state_bits=bits)
    t = wl.step
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        eager.step(t)
        graphed.step(t)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        graphed.step(t)
    torch.cuda.synchronize()
    names = ["master", "rank_sq"] + (["m", "v"] if bits == 32 else ["m8", "v8", "m_scale", "v_scale"])
    for rep in range(4):
        eager.fill_grads(wl.step + 10 + rep)
        graphed.fill_grads(wl.step + 10 + rep)
        torch.cuda.synchronize()
        eager.step(t)
        g.replay()
        torch.cuda.synchronize()
        for k in names:
            x, y = getattr(eager, k), getattr(graphed, k)
            x, y = (z.view(torch.uint8) for z in (x, y))
            assert torch.equal(x, y), (rep, k)
        for i in graphed.touched:
            assert torch.equal(graphed.params[i].view(torch.int16), eager.params[i].view(torch.int16)), (rep, i)


def test_list_made_while_capturing():
    """The table's upload is captured with the step and runs at each replay."""
    case = Case([700, 5, 300], 8, seed=3).to_device()
    twin = Case([700, 5, 300], 8, seed=3).to_device()
    sums = torch.full((1,), 0.25, dtype=torch.float64, device=DEV)
    hp = zero.hparams(step=2)
    views = {k: a.views for k, a in case.A.items()}
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lst = tensors.zero_tensors(views["param"], views["m"], views["v"], master=views["master"],
                                   m_scale=views["m_scale"], v_scale=views["v_scale"])
        tensors.zero_tensors_adamw_step(lst, case.grad_ptrs, hp, sums, 1)
    for _ in range(3):
        g.replay()
        tensors.zero_tensors_adamw_step(twin.list, twin.grad_ptrs, hp, sums, 1)
        torch.cuda.synchronize()
        for k in case.A:
            assert np.array_equal(case.A[k].bits(), twin.A[k].bits()), k


@pytest.mark.parametrize("bits", [32, 8])
def test_lists_on_several_streams_and_threads(bits):
    """Six lists, each stepped by a thread of its own on a stream of its own:
    as if one after another."""
    n = 6
    cases = [Case([40_000 + 17 * k, 3, 999], bits, seed=k).to_device() for k in range(n)]
    parts = np.full(4, 0.3)
    d_parts = torch.from_numpy(parts).to(DEV)
    ws = [torch.empty(tensors.zero_tensors_sqnorm_workspace_bytes(c.list) // 8, dtype=torch.float64, device=DEV)
          for c in cases]
    norms = torch.zeros(n, dtype=torch.float64, device=DEV)
    streams = [torch.cuda.Stream() for _ in range(n)]
    torch.cuda.synchronize()
    errors = []

    def work(k):
        try:
            st = streams[k] if k % 2 else streams[k].cuda_stream
            tensors.zero_tensors_sqnorm(cases[k].list, cases[k].grad_ptrs, norms[k:k + 1], False, ws[k], stream=st)
            tensors.zero_tensors_adamw_step(cases[k].list, cases[k].grad_ptrs, hp_of(O.AdamWHParams(), 5), d_parts, 4,
                                            stream=st)
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(k,)) for k in range(n)]
    [x.start() for x in threads]
    [x.join() for x in threads]
    torch.cuda.synchronize()
    assert not errors, errors
    coef = O.clip_coef(O.global_sqnorm(parts), 1.0)
    for k, c in enumerate(cases):
        want = sum(O.sqnorm_f32(g) for g in c.grads)
        assert abs(norms[k].item() - want) <= 1e-12 * want
        if bits == 32:
            check32(c, [O.AdamWHParams()], [5], coef, d_parts, 4)
        else:
            check8(c, [O.AdamWHParams()], [5], coef)


def test_a_list_dropped_while_its_step_runs():
    """The step waits on a side stream behind other work while its list is
    dropped and new tensors are allocated: its table is not given out again
    before the step has read it."""
    case, twin = (Case([70_000, 300], 8, seed=33).to_device() for _ in range(2))
    sums = torch.full((1,), 0.25, dtype=torch.float64, device=DEV)
    side = torch.cuda.Stream()
    busy = torch.randn(4096, 4096, device=DEV)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(20):
            busy = busy @ busy * 1e-3
        tensors.zero_tensors_adamw_step(case.list, case.grad_ptrs, zero.hparams(step=2), sums, 1)
    size = case.list.table.numel()
    case.list = None
    filled = [torch.full((size,), -1, dtype=torch.int64, device=DEV) for _ in range(8)]
    torch.cuda.synchronize()
    tensors.zero_tensors_adamw_step(twin.list, twin.grad_ptrs, zero.hparams(step=2), sums, 1)
    torch.cuda.synchronize()
    for k in case.A:
        assert np.array_equal(case.A[k].bits(), twin.A[k].bits()), k
    assert all(int(f.min()) == -1 for f in filled)


@pytest.mark.parametrize("bits", [32, 8])
def test_a_list_without_elements_or_gradients(bits):
    case = Case([0, 0, 5, 0], bits, seed=34, missing=(2,)).to_device()
    run_step(case)
    case.check_guards()
    untouched(case, 2)
    case = Case([0, 0], bits, seed=35).to_device()
    run_step(case)
    case.check_guards()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("lens", [[3_000_000, 5, 2_000_001], [1 << 20] * 9])
def test_long_lists(bits, lens):
    """Units of their own for the waves and whole rounds of XCD runs."""
    case = Case(lens, bits, seed=36).to_device()
    got = run_step(case)
    check32(case, *got, 4) if bits == 32 else check8(case, *got[:3])


def test_gradients_beyond_32_bit_offsets():
    """Two gradients 9 GB apart in bf16: more than 2^32 elements, so one launch cannot carry both."""
    arena = torch.empty(9_300_000_000, dtype=torch.uint8, device=DEV).view(torch.bfloat16)
    case = Case([3000, 2000, 1500], 8, seed=21).to_device()
    far = [arena[7:7 + 3000], arena[4_600_000_000:4_600_000_000 + 2000], arena[9000:9000 + 1500]]
    for a, b in zip(far, case.grad_list):
        a.copy_(b)
    case.grad_ptrs = zero.pointer_array(far)
    check8(case, *run_step(case)[:3])
    ws = torch.empty(tensors.zero_tensors_sqnorm_workspace_bytes(case.list) // 8, dtype=torch.float64, device=DEV)
    out = torch.zeros(1, dtype=torch.float64, device=DEV)
    tensors.zero_tensors_sqnorm(case.list, far, out, False, ws)
    want = sum(O.sqnorm_f32(g) for g in case.grads)
    assert abs(out.item() - want) <= 1e-12 * want


@pytest.mark.parametrize("bits", [32, 8])
def test_a_tensor_beyond_2_31_elements(bits):
    """Windows of whole blocks of a 2^31 + 70001-element tensor (its start,
    around 2^31, its end) get what a small list of the same windows gets."""
    n = (1 << 31) + 70_001
    wins = [(0, 5120), ((1 << 31) - 2560, (1 << 31) + 2560), ((1 << 31) + 65536, n)]

    def draw(dtype, std, positive=False):
        x = torch.empty(n, dtype=dtype, device=DEV)
        for lo in range(0, n, 1 << 28):
            part = torch.randn(min(1 << 28, n - lo), device=DEV).mul_(std)
            x[lo:lo + part.numel()] = part.abs_() if positive else part
        return x

    g, master = draw(torch.bfloat16, 1e-3), draw(torch.float32, 0.02)
    param = torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    if bits == 32:
        cols = {"m": draw(torch.float32, 1e-4), "v": draw(torch.float32, 1e-8, True)}
    else:
        nb = tensors.state8_blocks(n)
        cols = {k: torch.randint(0, 0x70, (n,), dtype=torch.uint8, device=DEV) for k in ("m", "v")}
        cols.update(m_scale=torch.rand(nb, device=DEV).mul_(1e-6), v_scale=torch.rand(nb, device=DEV).mul_(1e-6))

    def window(x, lo, hi):
        return x[lo // 256:-(-hi // 256)] if x.numel() < n else x[lo:hi]

    small = {k: [window(x, lo, hi).clone() for lo, hi in wins]
             for k, x in {"param": param, "master": master, "g": g, **cols}.items()}
    big = tensors.zero_tensors([param], [cols["m"]], [cols["v"]], master=[master],
                               **{k: [x] for k, x in cols.items() if "scale" in k})
    little = tensors.zero_tensors(small["param"], small["m"], small["v"], master=small["master"],
                                  **{k: small[k] for k in cols if "scale" in k})
    sums = torch.full((2,), 0.7, dtype=torch.float64, device=DEV)
    tensors.zero_tensors_adamw_step(big, [g], zero.hparams(step=4), sums, 2)
    tensors.zero_tensors_adamw_step(little, small["g"], zero.hparams(step=4), sums, 2)
    torch.cuda.synchronize()
    for k, x in {"param": param, "master": master, **cols}.items():
        for (lo, hi), y in zip(wins, small[k]):
            assert torch.equal(window(x, lo, hi).view(torch.uint8), y.view(torch.uint8)), (k, lo)
    ws = torch.empty(tensors.zero_tensors_sqnorm_workspace_bytes(big) // 8, dtype=torch.float64, device=DEV)
    out = torch.zeros(1, dtype=torch.float64, device=DEV)
    tensors.zero_tensors_sqnorm(big, [g], out, False, ws)
    want = sum(float(torch.dot(p, p)) for lo in range(0, n, 1 << 28) for p in [g[lo:lo + (1 << 28)].double()])
    assert abs(out.item() - want) <= 1e-11 * want


def test_binding_refusals_on_the_device():
    f = lambda n, t=torch.float32: torch.zeros(n, dtype=t, device=DEV)  # noqa: E731
    lst = tensors.zero_tensors([f(8)], [f(8)], [f(8)])
    ws, out = f(1, torch.float64), f(1, torch.float64)
    for bad, err in (([f(7)], ValueError), ([f(8, torch.bfloat16)], TypeError), ([f(8), f(8)], ValueError),
                     ([f(16)[::2]], ValueError), ([torch.zeros(8)], TypeError)):
        with pytest.raises(err):
            tensors.zero_tensors_sqnorm(lst, bad, out, False, ws)
    with pytest.raises(ValueError, match="sums of squares"):
        tensors.zero_tensors_adamw_step(lst, [f(8)], zero.hparams(), out, 2)
    with pytest.raises(ValueError, match="pointers"):
        tensors.zero_tensors_sqnorm(lst, zero.pointer_array([]), out, False, ws)
    with pytest.raises(zero.ZeroError, match="workspace"):
        tensors.zero_tensors_sqnorm(lst, [f(8)], out, False, ws, ws_bytes=0)
    with pytest.raises(zero.ZeroError, match="overlap"):
        x = f(8)
        tensors.zero_tensors([x], [x], [f(8)])
    with pytest.raises(zero.ZeroError, match="32-bit"):
        tensors.zero_tensors_state_export(lst, [f(8)], [f(8)])
    with pytest.raises(ValueError, match="m_scale"):
        tensors.zero_tensors([f(300)], [f(300, torch.uint8)], [f(300, torch.uint8)], m_scale=[f(1)], v_scale=[f(2)])
