"""The step over a list of tensors (include/zero_tensors.h) on the GPU:

  * the 32-bit step bit for bit against the flat update of the same values
    (zero_adamw_step_arrays) and against the oracle;
  * the 8-bit step against the fp64 definition (oracle.state8): every byte
    equal, masters within the derived fp32 bound;
  * the norm against exact sums, import and export against the definition.

Lists hold ragged tensors (0 to several thousand elements) at every phase,
with guard elements around each that must keep their bits.
"""

import numpy as np
import pytest

from fsdp_sharded_mixed_zero_amd import tensors, zero
from oracle import state8 as S8
from oracle import step as O
from devbits import hp_of
from tensor_lists import Case
from tolerance import assert_bf16_param, assert_f32_state

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda"
RAGGED = [1, 0, 2, 3, 4, 5, 7, 63, 64, 65, 255, 256, 257, 511, 513, 1000, 1023, 1024, 1025, 2047, 2049, 4099, 0, 6]


def many_lens(count=900, seed=4):
    return [int(n) for n in np.random.default_rng(seed).integers(0, 700, count)]


def sums(n_ranks, total, seed):
    parts = np.abs(np.random.default_rng(seed).standard_normal(n_ranks)) * total / n_ranks
    return parts, torch.from_numpy(parts).to(DEV)


def oracle_hps(groups, **over):
    kinds = [dict(), dict(weight_decay=0.0), dict(lr=3e-4, beta1=0.8, beta2=0.95, eps=1e-6)]
    return [O.AdamWHParams(**{**kinds[k % 3], **over}) for k in range(groups)]


def steps_of(groups, step):
    return [step + 7 * k for k in range(groups)]


def run_step(case, step=3, groups=1, n_ranks=4, total=2.0, seed=1, stream=None, pointers=True, **over):
    """One step of the case on the device; returns (hyperparameters, steps, coefficient)."""
    parts, d_parts = sums(n_ranks, total, seed)
    hps, steps = oracle_hps(groups, **over), steps_of(groups, step)
    tensors.zero_tensors_adamw_step(case.list, case.grad_ptrs if pointers else case.grad_list,
                                    [hp_of(h, s) for h, s in zip(hps, steps)], d_parts, n_ranks, stream)
    torch.cuda.synchronize()
    return hps, steps, O.clip_coef(O.global_sqnorm(parts), hps[0].max_norm, hps[0].clip_eps), d_parts


def untouched(case, i):
    """Tensor i has its old bits in every column."""
    for name, a in case.A.items():
        lo, hi = a.spans[i]
        assert np.array_equal(a.bits()[lo:hi], a.before[lo:hi]), (name, i)


# ------------------------------------------------------------------- 32 bits

def flat_twin(case, i, hp, step, d_parts, n_ranks):
    """zero_adamw_step_arrays on tensor i's values: (master, m, v, param bits)."""
    d = [torch.from_numpy(x[i].copy()).to(DEV) for x in (case.master, case.m, case.v)]
    g = torch.from_numpy(case.grad_bits[i].view(np.int16)).to(DEV).view(torch.bfloat16)
    out = torch.empty(case.lens[i], dtype=torch.bfloat16, device=DEV)
    zero.zero_adamw_step_arrays(g, *d, out, case.lens[i], hp_of(hp, step), d_parts, n_ranks)
    return [x.cpu().numpy() for x in d] + [out.view(torch.int16).cpu().numpy().view(np.uint16)]


def check32(case, hps, steps, coef, d_parts, n_ranks, twin=True):
    got = {k: a.tensors() for k, a in case.A.items()}
    masters = got["master"] if "master" in got else got["param"]
    case.check_guards()
    for i, n in enumerate(case.lens):
        if i in case.missing:
            untouched(case, i)
            continue
        if n == 0:
            continue
        hp, step = hps[case.group[i]], steps[case.group[i]]
        p, m, v, bits = O.adamw_step_f32grad(case.grads[i], case.master[i], case.m[i], case.v[i], step, hp, coef)
        assert_f32_state(masters[i], p, f"master {i}")
        assert_f32_state(got["m"][i], m, f"m {i}", case.m[i])
        assert_f32_state(got["v"][i], v, f"v {i}", case.v[i])
        if "master" in got:
            assert_bf16_param(got["param"][i], bits, p, f"param {i}", masters[i])
        if twin and case.grad_type == "bf16":
            flat = flat_twin(case, i, hp, step, d_parts, n_ranks)
            for name, a, b in zip(("master", "m", "v"), (masters[i], got["m"][i], got["v"][i]), flat):
                assert np.array_equal(a.view(np.uint32), b.view(np.uint32)), f"{name} {i} differs from the flat update"
            if "master" in got:
                assert np.array_equal(got["param"][i], flat[3])


@pytest.mark.parametrize("param", ["bf16", "f32"])
@pytest.mark.parametrize("grad", ["bf16", "f32"])
@pytest.mark.parametrize("align", [1, 64])
def test_step32_ragged(param, grad, align):
    case = Case(RAGGED, 32, param, grad, seed=align, missing=(4, 19), groups=3, align=align).to_device()
    check32(case, *run_step(case, groups=3), 4)


def test_step32_more_tensors_than_a_launch():
    case = Case(many_lens(), 32, seed=2, missing=range(0, 900, 11), groups=8).to_device()
    check32(case, *run_step(case, groups=8, n_ranks=70), 70, twin=False)


@pytest.mark.parametrize("step,over", [(1, {}), (1000, {}), (5, dict(max_norm=0.0)), (2, dict(eps=0.0))])
def test_step32_hyperparameters(step, over):
    case = Case([5000, 1, 300], 32, seed=step).to_device()
    check32(case, *run_step(case, step=step, pointers=False, **over), 4)


def test_step32_cancelled_masters_take_the_fp64_recompute():
    from cancellation_inputs import planted
    n = (1 << 18) + 77
    bits, master, m, v, step, G, deep, size = planted(n, 9, 1)
    case = Case([n], 32)
    case.grad_bits, case.master, case.m, case.v = [bits], [master], [m], [v]
    case.to_device()
    d = torch.tensor([G], dtype=torch.float64, device=DEV)
    tensors.zero_tensors_adamw_step(case.list, case.grad_ptrs, hp_of(O.AdamWHParams(), step), d, 1)
    flat = flat_twin(case, 0, O.AdamWHParams(), step, d, 1)
    for k, b in zip(("master", "m", "v", "param"), flat):
        assert np.array_equal(case.A[k].tensors()[0].view(b.dtype), b), k
    case.check_guards()


# -------------------------------------------------------------------- 8 bits

def check_codes(got, want, what):
    """Bytes and scales of one tensor. A scale may be one fp32 step from the
    definition's where the two fp64 evaluations of its maximum (a few 2^-53
    apart) fall on two sides of a rounding border; its block's bytes are then
    compared as the values they stand for."""
    for k in (1, 3):
        a, b = got[k].astype(np.float64), want[k].astype(np.float64)
        assert (np.abs(a - b) <= 2.0 ** -23 * np.abs(b)).all(), f"{what}: scale"
        off = np.repeat(a != b, S8.BLOCK)[:got[k - 1].size]
        assert np.array_equal(got[k - 1][~off] & 0x7F == S8.NAN, want[k - 1][~off] & 0x7F == S8.NAN), what
        number = (want[k - 1] & 0x7F != S8.NAN) & ~off
        assert np.array_equal(got[k - 1][number], want[k - 1][number]), f"{what}: {'m' if k == 1 else 'v'} bytes"
        assert off.mean() < 0.01 if off.size > 25600 else True


def check8(case, hps, steps, coef):
    got = {k: a.tensors() for k, a in case.A.items()}
    masters = got["master"] if "master" in got else got["param"]
    case.check_guards()
    for i, n in enumerate(case.lens):
        if i in case.missing:
            untouched(case, i)
            continue
        if n == 0:
            continue
        hp, step = hps[case.group[i]], steps[case.group[i]]
        p, m1, v1, codes = S8.adamw8_step(case.grads[i], case.master[i], *case.state[i], step, hp, coef)
        check_codes([got[k][i] for k in ("m", "m_scale", "v", "v_scale")], codes, f"tensor {i}")
        err = np.abs(masters[i].astype(np.float64) - p)
        assert (err <= S8.update_bound(case.master[i], m1, v1, step, hp)).all(), f"master {i}: {err.max()}"
        if "master" in got:
            cast = torch.from_numpy(masters[i].copy()).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)
            assert np.array_equal(got["param"][i], cast), f"param {i} is not the bf16 of its master"


@pytest.mark.parametrize("param", ["bf16", "f32"])
@pytest.mark.parametrize("grad", ["bf16", "f32"])
@pytest.mark.parametrize("align", [1, 64])
def test_step8_ragged(param, grad, align):
    case = Case(RAGGED, 8, param, grad, seed=align, missing=(4, 19), groups=3, align=align).to_device()
    check8(case, *run_step(case, groups=3)[:3])


def test_step8_more_tensors_than_a_launch():
    case = Case(many_lens(), 8, seed=2, missing=range(0, 900, 11), groups=8).to_device()
    check8(case, *run_step(case, groups=8, n_ranks=70)[:3])


def test_step8_a_million_elements():
    """2^20 elements: thousands of moments within 2^-20 of a border between two bytes, all decided as in fp64."""
    case = Case([1 << 20, 77], 8, seed=5).to_device()
    check8(case, *run_step(case, step=1000)[:3])


@pytest.mark.parametrize("step,over", [(1, {}), (1000, {}), (5, dict(max_norm=0.0)), (3, dict(beta1=0.0, beta2=0.0))])
def test_step8_hyperparameters(step, over):
    case = Case([5000, 1, 300], 8, seed=step).to_device()
    check8(case, *run_step(case, step=step, pointers=False, **over)[:3])


@pytest.mark.parametrize("scale", [1e-30, 3e-23, 1e-18, 1e-9, 1e6, 1e15])
def test_step8_magnitudes(scale):
    """Gradients and moments from the smallest whose square fp32 still holds to the largest."""
    case = Case([700, 256], 8, grad="f32", seed=7, m_std=scale, v_std=scale ** 2, g_std=scale).to_device()
    check8(case, *run_step(case, max_norm=0.0)[:3])


def test_step8_first_step_from_zeroed_state():
    case = Case([1000, 3], 8, seed=8, m_std=0.0, v_std=0.0)
    case.state = [tuple(np.zeros_like(x) for x in s) for s in case.state]
    case.grads[0][100:400] = 0.0
    case.grad_bits[0][100:400] = 0
    case.to_device()
    check8(case, *run_step(case, step=1)[:3])


def test_step8_wide_ranges_inside_a_block():
    """Moments over 30 binades in one block: underflowing bytes, and roots kept above zero."""
    rng = np.random.default_rng(9)
    case = Case([2048], 8, grad="f32", seed=9)
    case.grads = case.grad_bits = [(rng.standard_normal(2048) * 2.0 ** rng.uniform(-30, 0, 2048)).astype(np.float32)]
    case.state = [S8.encode(case.grads[0] * 0.3, case.grads[0].astype(np.float64) ** 2)]
    case.to_device()
    check8(case, *run_step(case)[:3])
    old, new = case.state[0][2], case.A["v"].tensors()[0]
    assert (new[(old > 0) | (case.grads[0] != 0)] > 0).all()


def test_step8_not_finite():
    """A NaN or infinite gradient spoils its own element: its neighbours get the bytes they would have without it."""
    case = Case([600, 300], 8, grad="f32", seed=10)
    for k, bad in ((5, np.nan), (290, np.inf), (599, -np.inf)):
        case.grads[0][k] = bad
    case.to_device()
    hps, steps, coef, _ = run_step(case, max_norm=0.0)
    p, m1, v1, codes = S8.adamw8_step(case.grads[0], case.master[0], *case.state[0], steps[0], hps[0], coef)
    got = {k: a.tensors()[0] for k, a in case.A.items()}
    check_codes([got[k] for k in ("m", "m_scale", "v", "v_scale")], codes, "tensor 0")
    assert np.isnan(got["master"][[5, 290, 599]]).all()
    fine = np.isfinite(case.grads[0])
    assert np.isfinite(got["master"][fine]).all()
    case.check_guards()


def test_step8_nan_norm_spoils_every_element():
    case = Case([300], 8, seed=11).to_device()
    tensors.zero_tensors_adamw_step(case.list, case.grad_ptrs, zero.hparams(step=2),
                                    torch.full((1,), float("nan"), dtype=torch.float64, device=DEV), 1)
    assert np.isnan(case.A["master"].tensors()[0]).all()
    assert (case.A["m"].tensors()[0] & 0x7F == S8.NAN).all() and (case.A["v"].tensors()[0] & 0x7F == S8.NAN).all()
    case.check_guards()


def test_step8_borders():
    """Second moments whose roots lie on, just below and just above the border of two bytes."""
    grid = S8.e4m3_table()[:127]
    mid = (grid[:-1] + grid[1:]) / 2
    root = np.concatenate([mid, mid * (1 - 2e-7), mid * (1 + 2e-7), [448.0]])
    v = np.concatenate([(root ** 2)[:255], [448.0 ** 2], (root ** 2)[255:], [448.0 ** 2]]).astype(np.float32)
    m = np.concatenate([root[:255], [448.0], -root[255:], [448.0]]).astype(np.float32)
    case = Case([v.size], 8).to_device()
    check_import(case, [m], [v])


# --------------------------------------------------------- import and export

def check_import(case, ms, vs, both=True):
    d = [[torch.from_numpy(np.ascontiguousarray(x)).to(DEV) for x in col] for col in (ms, vs)]
    tensors.zero_tensors_state_import(case.list, *d)
    got = {k: a.tensors() for k, a in case.A.items()}
    for i, n in enumerate(case.lens):
        if n:
            check_codes([got[k][i] for k in ("m", "m_scale", "v", "v_scale")],
                        S8.encode(ms[i].astype(np.float64), vs[i].astype(np.float64)), f"tensor {i}")
    for name in ("param", "master"):
        if name in case.A:
            assert np.array_equal(case.A[name].bits(), case.A[name].before), f"{name} changed"
    case.check_guards()


@pytest.mark.parametrize("lens", [RAGGED, many_lens()], ids=["ragged", "900"])
def test_import_and_export(lens):
    case = Case(lens, 8, seed=12).to_device()
    rng = np.random.default_rng(13)
    ms = [(rng.standard_normal(n) * 1e-3).astype(np.float32) for n in lens]
    vs = [(rng.random(n) ** 6 * 1e-6).astype(np.float32) for n in lens]
    check_import(case, ms, vs)
    out = [[torch.full((n + 2,), 7.0, device=DEV) for n in lens] for _ in range(2)]
    inner = [[x[1:-1] for x in col] for col in out]
    before = {k: a.bits() for k, a in case.A.items()}
    tensors.zero_tensors_state_export(case.list, *inner)
    for k, a in case.A.items():
        assert np.array_equal(a.bits(), before[k]), f"the export changed {k}"
    got = {k: a.tensors() for k, a in case.A.items()}
    for i, n in enumerate(lens):
        m, v = S8.decode(got["m"][i], got["m_scale"][i], got["v"][i], got["v_scale"][i])
        assert np.array_equal(inner[0][i].cpu().numpy(), m.astype(np.float32))
        # (S * scale)^2 in fp64 carries two roundings more than the definition's: at most one fp32 step
        v32 = v.astype(np.float32)
        assert (np.abs(inner[1][i].cpu().numpy().astype(np.float64) - v32) <= np.spacing(v32)).all()
        for x in (out[0][i], out[1][i]):
            assert x[0] == 7.0 and x[-1] == 7.0


def test_import_leaves_out_tensors_without_arrays():
    case = Case([300, 500, 0, 40], 8, seed=14).to_device()
    z = [torch.zeros(n, device=DEV) for n in case.lens]
    tensors.zero_tensors_state_import(case.list, [z[0], None, None, z[3]], [z[0], None, None, z[3]])
    untouched(case, 1)
    assert not case.A["m"].tensors()[0].any() and not case.A["v"].tensors()[3].any()


def test_import_of_negative_and_not_finite_moments():
    m = np.linspace(-1, 1, 300).astype(np.float32)
    v = np.linspace(0, 1, 300).astype(np.float32)
    m[3], m[4], v[5], v[6], v[7], v[8] = np.nan, np.inf, np.nan, np.inf, -1.0, -0.0
    check_import(Case([300], 8).to_device(), [m], [v])


# ------------------------------------------------------------------ the norm

@pytest.mark.parametrize("grad", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [RAGGED, many_lens(), [1], [0, 0], [300_000, 0, 5]], ids=["ragged", "900", "1", "0", "big"])
def test_sqnorm(lens, grad):
    case = Case(lens, 32, grad=grad, seed=15, missing=(3, 8) if len(lens) > 8 else (), g_std=0.3).to_device()
    want = sum(O.sqnorm_f32(g) for i, g in enumerate(case.grads) if i not in case.missing)
    ws = torch.full((tensors.zero_tensors_sqnorm_workspace_bytes(case.list) // 8,), float("nan"), dtype=torch.float64,
                    device=DEV)
    out = torch.full((3,), 5.0, dtype=torch.float64, device=DEV)
    for args in ((case.grad_ptrs,), (case.grad_list,)):
        ws.fill_(float("nan"))
        tensors.zero_tensors_sqnorm(case.list, *args, out[1:2], False, ws)
        first = out[1].item()
        # non-negative terms, each added at most once per level: n * 2^-53 relative covers any order
        assert abs(first - want) <= max(1, sum(lens)) * 2.0 ** -53 * want
        tensors.zero_tensors_sqnorm(case.list, *args, out[1:2], True, ws)
        assert out[1].item() == first + first
        assert out[0].item() == 5.0 and out[2].item() == 5.0
    case.check_guards()


def test_sqnorm_does_not_depend_on_where_the_tensors_lie():
    got = []
    for align in (1, 64):
        case = Case(RAGGED, 32, seed=16, align=align).to_device()
        ws = torch.empty(tensors.zero_tensors_sqnorm_workspace_bytes(case.list) // 8, dtype=torch.float64, device=DEV)
        out = torch.zeros(1, dtype=torch.float64, device=DEV)
        tensors.zero_tensors_sqnorm(case.list, case.grad_ptrs, out, False, ws)
        got.append(out.item())
    assert got[0] == got[1]
