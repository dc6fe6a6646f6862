"""The norm's gradient on both sides of every width at which its kernel takes more
threads, the same ones for both types, with more rows than one launch of blocks of
columns and rows takes."""

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from fsdp_sharded_mixed_zero_amd import layers

import layer_cases as C  # noqa: E402
from layer_cases import DEV, close, generator, normal, stored  # noqa: E402
from oracle import layers as O  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype,dim", [(BF16, d) for d in (1536, 1537, 2048, 2049, 2555, 2560, 2561, 4096, 4097, 5120, 5121, 6144, 6145)] +
                         [(F32, d) for d in (1024, 1025, 1277, 1280, 1281, 2048, 2049, 2560, 2561, 4096, 4097, 5120, 5121, 6144, 6145)])
@pytest.mark.parametrize("rms", [False, True])
def test_norm_grad_where_the_threads_change(dtype, dim, rms):
    n = 520 if dim > 4096 else 270
    gen = generator(dim)
    x = (normal(gen, n, dim) * (normal(gen, dim) * 0.5).exp() + 0.3).to(dtype)
    d_y, d_total, w = normal(gen, n, dim, dtype=dtype), normal(gen, n, dim, dtype=dtype), normal(gen, dim, dtype=BF16)
    _, mean, rstd = (torch.from_numpy(v).float().to(DEV) for v in O.norm(C.np64(x), rms=rms))
    d_x, d_w, d_b = torch.empty_like(x), torch.empty(dim, device=DEV), torch.empty(dim, device=DEV)
    ws = torch.full((layers.zero_norm_grad_workspace_bytes(n, dim) // 4,), float("nan"), device=DEV)
    layers.zero_norm_grad(d_y, x, mean, rstd, d_x, ws, weight=w, d_weight=d_w, d_bias=d_b, d_total=d_total, rms=rms)
    want, bound = C.norm_grad_want(d_y, x, mean, rstd, w, d_total, rms, dtype)
    close(d_x, want[0], bound[0], "d_x")
    for got, v, e, what in zip((d_w, d_b), want[1:], bound[1:], ("d_weight", "d_bias")):
        close(got, v, stored(e, v, F32), what)
