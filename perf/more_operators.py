"""Token tables and norms: the measured cases.

Four operators on the parameters that a rank holds apart from its matrices:

  embed       lookup in a token table: out[t] = scale * table[token[t]]
  embed_grad  its gradient by sorted tokens, for the whole table or for the part
              of it that lies in a rank's shard, written or added to what the
              micro-batches before left there
  norm        layer norm (or its form without mean and bias) of rows, the
              residual added before it in the same pass
  norm_grad   its gradient: of the rows, with the skip path's added, and of weight
              and bias, written or added

A token outside the table (-1: padding) reads as zeros and has no gradient.
``run`` computes them with elementary torch operations, or with the library's
calls where ``own`` is true.
"""

import math

import torch

own = False

SEQUENCE = 1024             # tokens of one sequence; in padded cases each ends early
EPS = 1e-5


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # the next tokens of eight sequences, GPT-2 1.5B's table: the latency end
        {"name": "embed gpt2-1.5b 8", "op": "embed", "n": 8, "rows": 50257, "dim": 1600, "ids": "i64", "table": "bf16",
         "out": "bf16", "scale": 1.0, "padded": False},
        # a micro-batch of 16 sequences through a 7B model's fp32 table, scaled by the root of its width
        {"name": "embed llama-7b 16x1024 f32", "op": "embed", "n": 16384, "rows": 32000, "dim": 4096, "ids": "i32",
         "table": "f32", "out": "bf16", "scale": 64.0, "padded": True},
        # half a sequence added to GPT-2 1.5B's fp32 accumulator
        {"name": "embed_grad gpt2-1.5b 512 add", "op": "embed_grad", "n": 512, "rows": 50257, "dim": 1600, "ids": "i64",
         "out": "bf16", "grad": "f32", "scale": 1.0, "padded": False, "part": 1, "accumulate": True},
        # eight sequences, the 7.5B model's whole bf16 gradient: most rows get none and are written as zeros
        {"name": "embed_grad gpt-7.5b 8x1024", "op": "embed_grad", "n": 8192, "rows": 50257, "dim": 2944, "ids": "i64",
         "out": "bf16", "grad": "bf16", "scale": 1.0, "padded": True, "part": 1, "accumulate": False},
        # the tokens of eight ranks' micro-batches on the 70B model, added to this rank's eighth of the table
        {"name": "embed_grad llama-70b/8 32x1024 add", "op": "embed_grad", "n": 32768, "rows": 32000, "dim": 8192,
         "ids": "i32", "out": "bf16", "grad": "f32", "scale": 1.0, "padded": False, "part": 8, "accumulate": True},
        # a small vocabulary, every size odd, fp32 throughout
        {"name": "embed_grad ragged f32", "op": "embed_grad", "n": 3001, "rows": 1009, "dim": 777, "ids": "i64", "out": "f32",
         "grad": "f32", "scale": 27.875, "padded": True, "part": 1, "accumulate": False},
        # eight rows between two of GPT-2 1.5B's layers at decoding
        {"name": "norm gpt2-1.5b 8", "op": "norm", "n": 8, "dim": 1600, "type": "bf16", "weight": "bf16", "rms": False,
         "residual": True},
        # a micro-batch of the 7.5B model before its MLP
        {"name": "norm gpt-7.5b 8x1024", "op": "norm", "n": 8192, "dim": 2944, "type": "bf16", "weight": "bf16", "rms": False,
         "residual": True},
        # the 70B model's norm over four long sequences, fp32 weights: the largest
        {"name": "norm llama-70b 4x4096 rms", "op": "norm", "n": 16384, "dim": 8192, "type": "bf16", "weight": "f32",
         "rms": True, "residual": False},
        # one sequence backward through a norm of GPT-2 1.5B, weight gradients added in fp32
        {"name": "norm_grad gpt2-1.5b 1024 add", "op": "norm_grad", "n": 1024, "dim": 1600, "type": "bf16", "weight": "bf16",
         "grad": "f32", "rms": False, "residual": True, "accumulate": True},
        # 16 sequences backward through a norm of the 7.5B model
        {"name": "norm_grad gpt-7.5b 16x1024", "op": "norm_grad", "n": 16384, "dim": 2944, "type": "bf16", "weight": "bf16",
         "grad": "bf16", "rms": False, "residual": True, "accumulate": False},
        # every size odd, fp32 throughout, without mean and bias
        {"name": "norm_grad ragged f32 rms", "op": "norm_grad", "n": 5003, "dim": 1111, "type": "f32", "weight": "f32",
         "grad": "f32", "rms": True, "residual": False, "accumulate": False},
    ]


MOST = 500_000_000          # bytes of a drawn case; the largest listed one moves 537 million


def draw(rng):
    """One more case: 1 to 32768 tokens or rows, widths from 64 to 8192, tables of 1000 to 60000 rows."""

    def spread(low, high):
        return round(math.exp(rng.uniform(math.log(low), math.log(high))))

    op = rng.choice(["embed", "embed_grad", "embed_grad", "norm", "norm_grad", "norm_grad"])
    dim = spread(64, 8192)
    if rng.random() < 0.6:
        dim = dim // 64 * 64
    case = {"op": op, "n": spread(1, 32768), "dim": dim}
    kind = lambda: rng.choice(["bf16", "bf16", "f32"])  # noqa: E731
    if op in ("embed", "embed_grad"):
        case.update(rows=rng.randint(1000, 60000), ids=rng.choice(["i64", "i32"]), out=kind(),
                    scale=rng.choice([1.0, 1.0, math.sqrt(dim), 0.1]), padded=rng.random() < 0.5)
        if op == "embed":
            case.update(table=kind())
        else:
            case.update(grad=kind(), part=rng.choice([1, 1, 2, 8, 64]), accumulate=rng.random() < 0.5)
    else:
        case.update(type=kind(), weight=kind(), rms=rng.random() < 0.4, residual=rng.random() < 0.5)
        if op == "norm_grad":
            case.update(grad=kind(), accumulate=rng.random() < 0.5)
    while work(case)["bytes"] > MOST:
        case["n"] = max(1, case["n"] * 3 // 4)
        if "rows" in case:
            case["rows"] = max(1000, case["rows"] * 3 // 4)
    return case


def size_of(kind):
    return {"bf16": 2, "f32": 4, "i32": 4, "i64": 8}[kind]


def type_of(kind):
    return {"bf16": torch.bfloat16, "f32": torch.float32, "i32": torch.int32, "i64": torch.int64}[kind]


def part_of(case):
    """The first element of the table's part and its length: equal cuts of the flat table, so rows are cut as well."""
    total, parts = case["rows"] * case["dim"], case["part"]
    each = -(-total // parts)
    first = each * (1 if parts > 1 else 0)
    return first, min(each, total - first)


def distinct(rows, n):
    """How many rows n tokens are expected to meet, for the distribution of tokens() below."""
    p = 1.0 / (torch.arange(rows, dtype=torch.float64) + 2.7)
    return float((1 - (1 - p / p.sum()) ** n).sum())


def work(case):
    n, dim, op = case["n"], case["dim"], case["op"]
    if op in ("embed", "embed_grad"):
        live = n * (0.75 if case["padded"] else 1.0)
        met = distinct(case["rows"], max(1, round(live)))
        rows = live * dim
        if op == "embed":
            return {"bytes": n * size_of(case["ids"]) + met * dim * size_of(case["table"]) + n * dim * size_of(case["out"]),
                    "flops": rows}
        share = part_of(case)[1] / (case["rows"] * dim)
        grad = 2 * met * dim * share if case["accumulate"] else case["rows"] * dim * share
        return {"bytes": n * size_of(case["ids"]) + rows * share * size_of(case["out"]) + grad * size_of(case["grad"]),
                "flops": rows * share}
    vectors = dim * (1 if case["rms"] else 2)
    stats = n * 4 * (1 if case["rms"] else 2)
    arrays = {"norm": 2 + 2 * case["residual"], "norm_grad": 3 + case["residual"]}[op]
    more = vectors * size_of(case["weight"])
    if op == "norm_grad":
        more = dim * size_of(case["weight"]) + vectors * size_of(case["grad"]) * (2 if case["accumulate"] else 1)
    return {"bytes": arrays * n * dim * size_of(case["type"]) + stats + more, "flops": n * dim * (8 if op == "norm" else 14)}


# ----------------------------------------------------------------- the inputs

def tokens(case, seed, dev):
    """Tokens as text has them: the k-th most frequent of them with a share of 1 / (k + 2.7), at any row of the table.
    In padded cases a sequence has half to all of its tokens, and -1 behind them. Drawn on the host: the same on any card."""
    gen = torch.Generator()
    gen.manual_seed(seed)
    n, rows = case["n"], case["rows"]
    up_to = (1.0 / (torch.arange(rows, dtype=torch.float64) + 2.7)).cumsum(0)
    rank = torch.searchsorted(up_to, torch.rand(n, generator=gen, dtype=torch.float64) * up_to[-1])
    t = torch.randperm(rows, generator=gen)[rank.clamp_(max=rows - 1)]
    if case["padded"]:
        each = min(SEQUENCE, n)
        length = torch.randint(each // 2, each + 1, (-(-n // each),), generator=gen)
        at = torch.arange(n)
        t = torch.where(at % each < length[at // each], t, -1)
    return t.to(type_of(case["ids"])).to(dev)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    n, dim, op = case["n"], case["dim"], case["op"]

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=gen, device=dev).mul_(std)

    s = {"case": case}
    if op in ("embed", "embed_grad"):
        s["tokens"] = tokens(case, seed, dev)
    if op == "embed":
        s["table"] = normal(case["rows"], dim, std=0.02).to(type_of(case["table"]))
        s["out"] = torch.empty(n, dim, dtype=type_of(case["out"]), device=dev)
    elif op == "embed_grad":
        s["first"], count = part_of(case)
        s["d_out"] = normal(n, dim, std=1e-3).to(type_of(case["out"]))
        s["grad"] = normal(count, std=1e-3).to(type_of(case["grad"]))
    else:
        # activations: channels of different sizes and means, a few of them far larger
        spread, mean = normal(dim).mul_(0.3).exp_(), normal(dim, std=0.2)
        spread[torch.randint(0, dim, (max(1, dim // 500),), generator=gen, device=dev)] *= 20.0
        kind, w_kind = type_of(case["type"]), type_of(case["weight"])
        s["x"] = (normal(n, dim) * spread + mean).to(kind)
        s["weight"] = (1.0 + normal(dim, std=0.1)).to(w_kind)
        s["bias"] = None if case["rms"] else normal(dim, std=0.1).to(w_kind)
        if op == "norm":
            s["residual"] = (normal(n, dim) * 2.0).to(kind) if case["residual"] else None
            s["total"] = torch.empty_like(s["x"]) if case["residual"] else None
            s["y"] = torch.empty_like(s["x"])
            s["mean"], s["rstd"] = (None if case["rms"] else torch.empty(n, device=dev)), torch.empty(n, device=dev)
        else:
            x = s["x"].double()
            m = torch.zeros(n, 1, dtype=torch.float64, device=dev) if case["rms"] else x.mean(1, keepdim=True)
            s["mean"] = None if case["rms"] else m[:, 0].float()
            s["rstd"] = ((x - m).square().mean(1) + EPS).rsqrt().float()
            s["d_y"] = normal(n, dim, std=1e-3).to(kind)
            s["d_total"] = normal(n, dim, std=1e-3).to(kind) if case["residual"] else None
            s["d_x"] = torch.empty_like(s["x"])
            g_kind = type_of(case["grad"])
            s["d_weight"] = normal(dim, std=1e-3).to(g_kind)
            s["d_bias"] = None if case["rms"] else normal(dim, std=1e-3).to(g_kind)
    if own:
        from fsdp_sharded_mixed_zero_amd import layers

        # scratch that a program keeps from step to step
        if op == "embed_grad":
            s["order"] = torch.empty(layers.zero_token_order_bytes(n, case["rows"]) // 4, dtype=torch.int32, device=dev)
            need = layers.zero_embedding_grad_workspace_bytes(n, dim)
            s["ws"] = torch.empty(need // 4, dtype=torch.float32, device=dev)
        elif op == "norm_grad":
            s["ws"] = torch.empty(layers.zero_norm_grad_workspace_bytes(n, dim) // 4, dtype=torch.float32, device=dev)
    return s


# ------------------------------------------------------------------- one pass

def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        from fsdp_sharded_mixed_zero_amd import layers

        s = state
        if op == "embed":
            layers.zero_embedding(s["tokens"], s["table"], s["out"], scale=case["scale"])
        elif op == "embed_grad":
            layers.zero_token_order(s["tokens"], case["rows"], s["order"])
            layers.zero_embedding_grad(s["order"], case["rows"], s["d_out"], s["grad"], s["ws"], scale=case["scale"],
                                       first=s["first"], accumulate=case["accumulate"])
        elif op == "norm":
            layers.zero_norm(s["x"], s["y"], s["mean"], s["rstd"], weight=s["weight"], bias=s["bias"], eps=EPS,
                             residual=s["residual"], total=s["total"], rms=case["rms"])
        else:
            layers.zero_norm_grad(s["d_y"], s["x"], s["mean"], s["rstd"], s["d_x"], s["ws"], weight=s["weight"],
                                  d_weight=s["d_weight"], d_bias=s["d_bias"], d_total=s["d_total"],
                                  accumulate=case["accumulate"], rms=case["rms"])
    else:
        {"embed": plain_embed, "embed_grad": plain_embed_grad, "norm": plain_norm, "norm_grad": plain_norm_grad}[op](state)
    keys = {"embed": ("out",), "embed_grad": ("grad",), "norm": ("y", "total", "mean", "rstd"),
            "norm_grad": ("d_x", "d_weight", "d_bias")}[op]
    return {k: state[k] for k in keys if state[k] is not None}


def plain_embed(s):
    t, rows = s["tokens"].long(), s["case"]["rows"]
    inside = (t >= 0) & (t < rows)
    out = s["table"][t.clamp(0, rows - 1)].float() * s["case"]["scale"]
    s["out"].copy_(out * inside[:, None])


def plain_embed_grad(s):
    case, dim = s["case"], s["case"]["dim"]
    first, count = s["first"], s["grad"].numel()
    low, high = first // dim, -(-(first + count) // dim)         # the rows that the part touches
    t = s["tokens"].long()
    t = torch.where((t >= low) & (t < high), t - low, high - low)        # all others: one row more, left out
    total = torch.zeros(high - low + 1, dim, dtype=torch.float32, device=t.device)
    total.index_add_(0, t, s["d_out"].float())
    new = total.view(-1)[first - low * dim:first - low * dim + count] * case["scale"]
    s["grad"].copy_(new + s["grad"].float() if case["accumulate"] else new)


def plain_norm(s):
    x, rms = s["x"].float(), s["case"]["rms"]
    if s["residual"] is not None:
        s["total"].copy_(x + s["residual"].float())
        x = s["total"].float()              # what the next layers read, and the gradient
    if not rms:
        mean = x.mean(1, keepdim=True)
        s["mean"].copy_(mean[:, 0])
        x = x - mean
    rstd = torch.rsqrt((x * x).mean(1, keepdim=True) + EPS)
    s["rstd"].copy_(rstd[:, 0])
    y = x * rstd * s["weight"].float()
    s["y"].copy_(y if rms else y + s["bias"].float())


def plain_norm_grad(s):
    case, x, dy = s["case"], s["x"].float(), s["d_y"].float()
    if not case["rms"]:
        x = x - s["mean"][:, None]
    x = x * s["rstd"][:, None]
    g = dy * s["weight"].float()
    dx = g - x * (g * x).mean(1, keepdim=True)
    if not case["rms"]:
        dx = dx - g.mean(1, keepdim=True)
    dx = dx * s["rstd"][:, None]
    s["d_x"].copy_(dx if s["d_total"] is None else dx + s["d_total"].float())
    for out, new in ((s["d_weight"], (dy * x).sum(0)), (s["d_bias"], None if case["rms"] else dy.sum(0))):
        if out is not None:
            out.copy_(new + out.float() if case["accumulate"] else new)


# -------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    wide = {k: v.double() for k, v in s.items() if torch.is_tensor(v) and v.is_floating_point()}
    if op == "embed":
        at = s["tokens"].long()
        out = torch.zeros(case["n"], case["dim"], dtype=torch.float64, device=at.device)
        live = torch.nonzero(at >= 0)[:, 0]
        out[live] = torch.index_select(wide["table"], 0, at[live]).mul_(case["scale"])
        return {"out": out}
    if op == "embed_grad":
        at = s["tokens"].long()
        live = torch.nonzero(at >= 0)[:, 0]
        out = torch.zeros(case["rows"], case["dim"], dtype=torch.float64, device=at.device)
        out.index_put_((at[live],), wide["d_out"][live] * case["scale"], accumulate=True)
        out = out.flatten()[s["first"]:s["first"] + s["grad"].numel()]
        return {"grad": out + wide["grad"] if case["accumulate"] else out}
    # a row's deviation is taken from the values that the operator reads: a residual's sum as it is stored
    x = wide["x"]
    total = None
    if op == "norm" and case["residual"]:
        total = x + wide["residual"]
        x = total.to(s["x"].dtype).double()
    bias = torch.zeros(case["dim"], dtype=torch.float64, device=x.device) if case["rms"] else wide["bias"]
    weight = wide["weight"]
    with torch.enable_grad():
        for v in (x, weight, bias):
            v.requires_grad_(op == "norm_grad")
        mean = torch.zeros_like(x[:, :1]) if case["rms"] else x.sum(1, keepdim=True) / case["dim"]
        rstd = (((x - mean) ** 2).sum(1, keepdim=True) / case["dim"] + EPS) ** -0.5
        y = (x - mean) * rstd * weight + bias
        if op == "norm":
            out = {"y": y, "total": total, "mean": None if case["rms"] else mean[:, 0], "rstd": rstd[:, 0]}
            return {k: v for k, v in out.items() if v is not None}
        dx, dw, db = torch.autograd.grad(y, (x, weight, bias), wide["d_y"])
    if case["residual"]:
        dx = dx + wide["d_total"]
    if case["accumulate"]:
        dw = dw + wide["d_weight"]
        db = db if case["rms"] else db + wide["d_bias"]
    return {"d_x": dx, "d_weight": dw} if case["rms"] else {"d_x": dx, "d_weight": dw, "d_bias": db}
