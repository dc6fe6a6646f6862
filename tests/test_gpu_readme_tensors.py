"""The README's tensor-list example, run as written on ragged tensors in two
groups, against the oracle of the 8-bit state."""

import os
import re
import textwrap

import numpy as np
import pytest

from fsdp_sharded_mixed_zero_amd import synth, zero
from oracle import state8 as S8
from oracle import step as O
from test_gpu_tensors import check_codes

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def example():
    text = open(README, encoding="utf-8").read()
    blocks = re.findall(r"(?:^    .*\n|^\n)+", text, re.M)
    code = [textwrap.dedent(b) for b in blocks if "zero_tensors_adamw_step" in b]
    assert len(code) == 1
    return code[0]


def test_readme_tensor_list_example():
    lens, groups, n_d, rank = [5000, 1, 768, 70_001], [0, 1, 1, 0], 3, 2
    rng = np.random.default_rng(12)
    bits = [synth.to_bf16_bits((rng.standard_normal(n) * 1e-3).astype(np.float32)) for n in lens]
    host = [(rng.standard_normal(n) * 0.02).astype(np.float32) for n in lens]
    bf16 = lambda b: torch.from_numpy(b.view(np.int16)).cuda().view(torch.bfloat16)  # noqa: E731
    hps = [O.AdamWHParams(weight_decay=wd, max_norm=1.0) for wd in (0.01, 0.0)]
    one = [zero.hparams(lr=h.lr, beta1=h.beta1, beta2=h.beta2, eps=h.eps, weight_decay=h.weight_decay,
                        max_norm=h.max_norm, clip_eps=h.clip_eps, step=1) for h in hps]
    rank_sq = torch.tensor([0.5, 0.25, 0.0], dtype=torch.float64, device="cuda")
    ns = {"torch": torch, "zero": zero, "params": [bf16(b) for b in bits], "grads": [bf16(b) for b in bits],
          "masters": [torch.from_numpy(h.copy()).cuda() for h in host], "groups": groups, "decay": one[0],
          "no_decay": one[1], "rank_sq": rank_sq, "rank": rank, "n_d": n_d}
    exec(example(), ns)  # noqa: S102 - the README's own code
    torch.cuda.synchronize()

    grads = [(b.astype(np.uint32) << 16).view(np.float32) for b in bits]
    own = float(rank_sq[rank])
    exact = sum(float((g.astype(np.float64) ** 2).sum()) for g in grads)
    assert own == pytest.approx(exact, rel=1e-12)      # 75 thousand positive terms, each rounding under 2^-53
    coef = O.clip_coef(O.global_sqnorm([0.5, 0.25, own]), 1.0, hps[0].clip_eps)
    for i, n in enumerate(lens):
        hp, blocks = hps[groups[i]], -(-n // 256)
        zeros = np.zeros(n, np.uint8), np.zeros(blocks, np.float32)
        p, m1, v1, codes = S8.adamw8_step(grads[i], host[i], *zeros, *zeros, 1, hp, coef)
        got = [ns[k][i].cpu().numpy() for k in ("m", "m_scale", "v", "v_scale")]
        check_codes(got, codes, f"tensor {i}")
        master = ns["masters"][i].cpu().numpy()
        assert (np.abs(master.astype(np.float64) - p) <= S8.update_bound(host[i], m1, v1, 1, hp)).all()
        cast = torch.from_numpy(master).to(torch.bfloat16)
        assert torch.equal(ns["params"][i].cpu().view(torch.int16), cast.view(torch.int16))
