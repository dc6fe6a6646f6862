"""The tensor-list calls on the host: every declared symbol is exported and
bound, constants and the record agree with the header, and every refusal the
header names is made before anything is enqueued. Addresses are made up: no
call here reaches a launch."""

import ctypes
import os
import re

import pytest

from fsdp_sharded_mixed_zero_amd import tensors, zero

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "zero_tensors.h")

pytestmark = pytest.mark.skipif(not os.path.exists(zero.LIB_PATH),
                                reason="libzero_mi355x.so not built (run __graft_entry__.build())")

BASE = 1 << 40


def header():
    return re.sub(r"/\*.*?\*/", "", open(HEADER, encoding="utf-8").read(), flags=re.S)


def test_declared_symbols_are_exported_and_bound():
    names = sorted(set(re.findall(r"\b(zero_tensors[a-z0-9_]*)\s*\(", header())))
    assert len(names) == 9, names
    for name in names:
        assert hasattr(tensors.library(), name)
        assert callable(getattr(tensors, name))
    assert set(names) == set(tensors._SIGNATURES)


def test_constants_and_record_agree_with_the_header():
    text = header()
    for name in ("ZERO_BF16", "ZERO_F32", "ZERO_STATE8_BLOCK", "ZERO_TENSOR_GROUPS", "ZERO_TENSORS_PER_LAUNCH"):
        assert int(re.search(rf"#define {name} (\d+)", text)[1]) == getattr(tensors, name), name
    fields = re.search(r"typedef struct \{(.*?)\} zero_tensor;", text, re.S)[1]
    assert re.findall(r"(\w+);", fields) == [f for f, _ in tensors.zero_tensor._fields_]
    assert ctypes.sizeof(tensors.zero_tensor) == 64


def record(k=0, n=1000, bits=8, kind=tensors.ZERO_BF16, **over):
    """Tensor k of a made-up list: buffers 1 MiB apart."""
    at = lambda j: BASE + (8 * k + j) * (1 << 20)  # noqa: E731
    r = dict(param=at(0), master=at(1) if kind == tensors.ZERO_BF16 else None, m=at(2), v=at(3),
             m_scale=at(4) if bits == 8 else None, v_scale=at(5) if bits == 8 else None, len=n, group=0)
    r.update(over)
    return r


def make(records, bits=8, param=tensors.ZERO_BF16, grad=tensors.ZERO_BF16, n=None):
    arr = (tensors.zero_tensor * max(1, len(records)))(*[tensors.zero_tensor(**r) for r in records])
    h = ctypes.c_void_p()
    rc = tensors.library().zero_tensors(arr, len(records) if n is None else n, param, grad, bits, ctypes.byref(h))
    return rc, h


def refused(rc, word):
    assert rc == zero.ZERO_EINVAL
    assert word in zero.zero_last_error(), zero.zero_last_error()


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("param", [tensors.ZERO_BF16, tensors.ZERO_F32])
def test_good_lists(bits, param):
    rs = [record(k, n, bits, param) for k, n in enumerate([1000, 1, 0, 4097])]
    rs[2] = dict(len=0, group=3)                       # no elements: no pointers needed
    rc, h = make(rs, bits, param)
    assert rc == zero.ZERO_OK
    lib = tensors.library()
    assert lib.zero_tensors_table_bytes(h) >= 4 * 64
    assert lib.zero_tensors_sqnorm_workspace_bytes(h) >= 8
    lib.zero_tensors_free(h)


def test_list_refusals():
    L = tensors.library()
    refused(make([record()], n=0)[0], "n must be")
    refused(make([record()], n=-3)[0], "n must be")
    refused(make([record()], n=(1 << 24) + 1)[0], "n must be")
    refused(make([record()], bits=16)[0], "state_bits")
    refused(make([record()], param=2)[0], "type")
    refused(make([record()], grad=-1)[0], "type")
    refused(make([record(n=-1)])[0], "length")
    refused(make([record(n=(1 << 40) + 1)])[0], "length")
    refused(make([record(k, n=1 << 39) for k in range(3)])[0], "length")
    refused(make([record(group=8)])[0], "group")
    refused(make([record(group=-1)])[0], "group")
    for name in ("param", "master", "m", "v", "m_scale", "v_scale"):
        refused(make([record(**{name: None})])[0], name)
        if name not in ("m", "v"):
            refused(make([record(**{name: BASE + (1 << 30) + 1})])[0], "misaligned")
    for name in ("m", "v"):
        refused(make([record(bits=32, **{name: BASE + (1 << 30) + 2})], bits=32)[0], "misaligned")
    refused(make([record()], param=tensors.ZERO_F32)[0], "master")
    refused(make([record()], bits=32)[0], "scales")
    refused(make([record(0), record(0)])[0], "overlap")                    # the same tensor twice
    refused(make([record(0), record(1, m=BASE + 2 * (1 << 20) + 999)])[0], "overlap")
    refused(make([record(0, m_scale=BASE + 5 * (1 << 20) + 12)])[0], "overlap")   # 4 scales of 4 bytes
    assert make([record(0, m_scale=BASE + 5 * (1 << 20) + 16)])[0] == zero.ZERO_OK
    h = ctypes.c_void_p()
    refused(L.zero_tensors(None, 1, 0, 0, 8, ctypes.byref(h)), "NULL")
    refused(L.zero_tensors((tensors.zero_tensor * 1)(), 1, 0, 0, 8, None), "NULL")
    assert L.zero_tensors_table_bytes(None) == 0 and L.zero_tensors_sqnorm_workspace_bytes(None) == 0
    L.zero_tensors_free(None)


def pointers(*p):
    return (ctypes.c_void_p * len(p))(*p)


def test_upload_and_norm_refusals():
    L = tensors.library()
    _, h = make([record(0), record(1)])
    need = L.zero_tensors_table_bytes(h)
    far = BASE + (1 << 36)
    refused(L.zero_tensors_upload(None, far, need, None), "NULL")
    refused(L.zero_tensors_upload(h, None, need, None), "NULL")
    refused(L.zero_tensors_upload(h, far + 8, need, None), "aligned")
    refused(L.zero_tensors_upload(h, far, need - 1, None), "need")
    refused(L.zero_tensors_upload(h, BASE + 64, need, None), "overlaps")
    g = pointers(far, far + 4096)
    ws = L.zero_tensors_sqnorm_workspace_bytes(h)
    ok = [h, g, far, 0, far + 512, ws, None]
    for k, value, word in ((0, None, "NULL"), (1, None, "NULL"), (2, None, "NULL"), (4, None, "NULL"),
                           (2, far + 4, "aligned"), (4, far + 4, "aligned"), (5, ws - 1, "workspace"),
                           (1, pointers(far + 1, far), "misaligned")):
        refused(L.zero_tensors_sqnorm(*ok[:k], value, *ok[k + 1:]), word)
    refused(L.zero_tensors_sqnorm(*ok), "no table")
    L.zero_tensors_free(h)


def step_call(h, g, groups, n_groups=None, sums=BASE + (1 << 37), ranks=4):
    arr = tensors.group_array(groups)
    return tensors.library().zero_tensors_adamw_step(h, g, arr, len(arr) if n_groups is None else n_groups, sums, ranks,
                                                     None)


def test_step_refusals():
    L = tensors.library()
    _, h = make([record(0), record(1, group=1)], grad=tensors.ZERO_F32)
    far = BASE + (1 << 36)
    g = pointers(far, far + 8192)
    hp = [zero.hparams(), zero.hparams(weight_decay=0.0)]
    refused(step_call(None, g, hp), "NULL")
    refused(step_call(h, None, hp), "NULL")
    refused(L.zero_tensors_adamw_step(h, g, None, 2, far, 4, None), "NULL")
    refused(step_call(h, g, hp, 0), "groups")
    refused(step_call(h, g, hp * 5), "groups")
    refused(step_call(h, g, hp[:1]), "uses group 1")
    refused(step_call(h, g, hp, sums=None), "sums of squares")
    refused(step_call(h, g, hp, ranks=0), "sums of squares")
    refused(step_call(h, g, hp, sums=far + 4), "misaligned")
    refused(step_call(h, g, [hp[0], zero.hparams(max_norm=2.0)]), "differ")
    refused(step_call(h, g, [hp[0], zero.hparams(clip_eps=2.0)]), "differ")
    for bad in (dict(lr=-1.0), dict(beta1=1.0), dict(beta2=-0.1), dict(eps=float("nan")), dict(weight_decay=-1.0),
                dict(step=0), dict(clip_eps=-1.0), dict(max_norm=float("nan"))):
        assert step_call(h, g, [hp[0], zero.hparams(**bad)]) == zero.ZERO_EINVAL, bad
    refused(step_call(h, pointers(far + 2, far), hp), "misaligned")
    refused(step_call(h, pointers(BASE + 1996, far), hp), "overlaps")   # the parameter's last bytes
    refused(step_call(h, pointers(BASE + 2 * (1 << 20) - 4 * 999, far), hp), "overlaps")   # ends in m's first bytes
    refused(step_call(h, pointers(None, BASE + 10 * (1 << 20)), hp), "overlaps")
    off = [zero.hparams(max_norm=0.0)] * 2
    for args in ((g, hp), (pointers(None, None), hp), (pointers(BASE + 2 * (1 << 20) - 4000, far), hp)):
        refused(step_call(h, *args), "no table")
    refused(step_call(h, g, off, sums=None, ranks=0), "no table")
    L.zero_tensors_free(h)


def test_state8_refusals():
    L = tensors.library()
    _, wide = make([record(bits=32)], bits=32)
    _, h = make([record(0), record(1)])
    far = BASE + (1 << 36)
    m, v = pointers(far, far + 4000), pointers(far + 8000, far + 12000)
    for fn in (L.zero_tensors_state_import, L.zero_tensors_state_export):
        refused(fn(None, m, v, None), "NULL")
        refused(fn(h, None, v, None), "NULL")
        refused(fn(h, m, None, None), "NULL")
        refused(fn(wide, m, v, None), "32-bit")
        refused(fn(h, pointers(None, far), v, None), "NULL")
        refused(fn(h, pointers(far + 2, far + 4004), v, None), "misaligned")
        refused(fn(h, pointers(BASE + 2 * (1 << 20) - 3996, far), v, None), "overlaps a buffer")
        refused(fn(h, m, v, None), "no table")
        refused(fn(h, pointers(None, far), pointers(None, far + 8000), None), "no table")
    refused(L.zero_tensors_state_export(h, m, pointers(far + 3996, far + 12000), None), "two exported")
    refused(L.zero_tensors_state_import(h, m, m, None), "no table")       # read only: may be shared
    L.zero_tensors_free(h)
    L.zero_tensors_free(wide)


def test_binding_refuses_what_the_library_cannot_see():
    torch = pytest.importorskip("torch")
    f = lambda n, t=torch.float32: torch.zeros(n, dtype=t)  # noqa: E731
    with pytest.raises(TypeError, match="device memory"):
        tensors.zero_tensors([f(8)], [f(8)], [f(8)])
    with pytest.raises(TypeError, match="bfloat16 or float32"):
        tensors.zero_tensors([f(8, torch.float16)], [f(8)], [f(8)])
    with pytest.raises(ValueError, match="at least one"):
        tensors.zero_tensors([], [], [])
    assert [tensors.state8_blocks(n) for n in (0, 1, 256, 257)] == [0, 1, 1, 2]
