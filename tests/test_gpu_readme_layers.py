"""The README's token-table and norm example, run as written, against the fp64 oracle."""

import os
import re
import textwrap

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import layer_cases as C  # noqa: E402
from layer_cases import DEV, U, close, generator, normal, stored  # noqa: E402
from oracle import layers as O  # noqa: E402

README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def example():
    text = open(README, encoding="utf-8").read()
    blocks = re.findall(r"(?:^    .*\n|^\n)+", text, re.M)
    code = [textwrap.dedent(b) for b in blocks if "zero_embedding_grad(" in b]
    assert len(code) == 1
    return code[0]


def test_readme_layers_example():
    n, rows, dim = 300, 70, 96
    gen = generator(31)
    bf16, f32 = torch.bfloat16, torch.float32
    old = [normal(gen, dim), normal(gen, dim), normal(gen, rows * dim)]
    ns = {"torch": torch, "n": n, "rows": rows, "dim": dim, "tokens": C.draw_tokens(n, rows, 1),
          "table": normal(gen, rows, dim, dtype=bf16), "weight": normal(gen, dim, dtype=bf16),
          "bias": normal(gen, dim, dtype=bf16), "d_y": normal(gen, n, dim, dtype=bf16)}
    ns["d_weight"], ns["d_bias"], ns["table_grad"] = (t.clone() for t in old)
    exec(example(), ns)  # noqa: S102 - the README's own code
    torch.cuda.synchronize()
    assert (C.np64(ns["h"]) == O.embedding(ns["tokens"].cpu().numpy(), C.np64(ns["table"]))).all()
    want, bound = C.norm_bounds(ns["h"], ns["weight"], ns["bias"], 1e-5, False, bf16)
    for got, v, e, what in zip((ns["y"], ns["mean"], ns["rstd"]), want, bound, ("y", "mean", "rstd")):
        close(got, v, e, what)
    want, bound = C.norm_grad_want(ns["d_y"], ns["h"], ns["mean"], ns["rstd"], ns["weight"], None, False, bf16)
    close(ns["d_h"], want[0], bound[0], "d_h")
    for got, v, e, before, what in zip((ns["d_weight"], ns["d_bias"]), want[1:], bound[1:], old, ("d_weight", "d_bias")):
        v = v + C.np64(before)
        close(got, v, stored(e + U * abs(v), v, f32), what)
    v, e = C.embedding_grad_want(ns["tokens"], ns["d_h"], rows, 1.0, old[2])
    close(ns["table_grad"].view(rows, dim), v, stored(e, v, f32), "table_grad")
