"""Lists of tensors for the tensor-list tests: every buffer of a list lies in
one arena per column (param, master, m, ...), at chosen element offsets, with
guard elements between the tensors that must keep their bits."""

import numpy as np

from fsdp_sharded_mixed_zero_amd import synth, tensors
from oracle import state8 as S8

DEV = "cuda"
GUARD = 3                       # elements between neighbours: an odd number, so that starts take every phase
FILL = {2: 0x7FA5, 4: 0x7FC0DEAD, 1: 0xA5}


def _torch_type(dtype):
    import torch
    return {"bf16": torch.bfloat16, "f32": torch.float32, "u8": torch.uint8}[dtype]


class Arena:
    """One column: tensors of the given lengths packed with GUARD elements
    before, between and after."""

    def __init__(self, values, dtype, align=1):
        import torch
        self.size = {"bf16": 2, "f32": 4, "u8": 1}[dtype]
        kind = {2: np.uint16, 4: np.uint32, 1: np.uint8}[self.size]
        at, self.spans = GUARD, []
        for x in values:
            at = -(-at // align) * align
            self.spans.append((at, at + x.size))
            at += x.size + GUARD
        host = np.full(at, FILL[self.size], kind)
        for (a, b), x in zip(self.spans, values):
            host[a:b] = np.ascontiguousarray(x).view(kind)
        self.before = host.copy()
        signed = {2: np.int16, 4: np.int32, 1: np.uint8}[self.size]
        self.flat = torch.from_numpy(host.view(signed)).to(DEV).view(_torch_type(dtype))
        self.views = [self.flat[a:b] for a, b in self.spans]
        self.kind, self.signed = kind, signed

    def bits(self):
        import torch
        t = self.flat.view({2: torch.int16, 4: torch.int32, 1: torch.uint8}[self.size])
        return t.cpu().numpy().view(self.kind)

    def check_guards(self, what):
        now = self.bits()
        inside = np.zeros(now.size, bool)
        for a, b in self.spans:
            inside[a:b] = True
        assert np.array_equal(now[~inside], self.before[~inside]), f"{what}: bytes outside the tensors changed"

    def tensors(self):
        b = self.bits()
        out = [b[lo:hi] for lo, hi in self.spans]
        return [x.view(np.float32) for x in out] if self.size == 4 else out


class Case:
    """Random inputs of a list: ``lens``, the types, the state. ``missing``:
    indices without a gradient. ``align``: 1 packs at odd phases, 64 starts
    every tensor on a boundary."""

    def __init__(self, lens, bits=32, param="bf16", grad="bf16", seed=0, missing=(), groups=1, align=1, m_std=1e-4,
                 v_std=1e-8, g_std=1e-3):
        rng = np.random.default_rng(seed)
        self.lens, self.bits, self.param_type, self.grad_type = list(lens), bits, param, grad
        self.group = [int(rng.integers(0, groups)) for _ in self.lens]
        normal = lambda n, std: (rng.standard_normal(n) * std).astype(np.float32)  # noqa: E731
        self.master = [normal(n, 0.02) for n in self.lens]
        self.grads = [normal(n, g_std) for n in self.lens]
        if grad == "bf16":
            self.grad_bits = [synth.to_bf16_bits(g) for g in self.grads]
            self.grads = [(b.astype(np.uint32) << 16).view(np.float32) for b in self.grad_bits]
        else:
            self.grad_bits = self.grads
        self.missing = set(missing)
        self.m = [normal(n, m_std) for n in self.lens]
        self.v = [np.abs(normal(n, v_std)) for n in self.lens]
        if bits == 8:
            self.state = [S8.encode(m, v) for m, v in zip(self.m, self.v)]
        self.align = align

    def to_device(self):
        from fsdp_sharded_mixed_zero_amd import zero
        al = self.align
        self.A = {"grad": Arena(self.grad_bits, self.grad_type, al)}
        if self.param_type == "bf16":
            self.A["param"] = Arena([np.full(n, 0x1234, np.uint16) for n in self.lens], "bf16", al)
            self.A["master"] = Arena(self.master, "f32", al)
        else:
            self.A["param"] = Arena(self.master, "f32", al)
        if self.bits == 32:
            self.A["m"], self.A["v"] = Arena(self.m, "f32", al), Arena(self.v, "f32", al)
        else:
            for name, k, kind in (("m", 0, "u8"), ("m_scale", 1, "f32"), ("v", 2, "u8"), ("v_scale", 3, "f32")):
                self.A[name] = Arena([s[k] for s in self.state], kind, al)
        views = lambda k: self.A[k].views if k in self.A else None  # noqa: E731
        import torch
        self.list = tensors.zero_tensors(views("param"), views("m"), views("v"), master=views("master"),
                                         m_scale=views("m_scale"), v_scale=views("v_scale"), group=self.group,
                                         grad_dtype=torch.bfloat16 if self.grad_type == "bf16" else torch.float32)
        self.grad_list = [None if i in self.missing else g for i, g in enumerate(self.A["grad"].views)]
        self.grad_ptrs = zero.pointer_array([g if g is not None and n else None
                                             for g, n in zip(self.grad_list, self.lens)])
        return self

    def check_guards(self):
        for name, a in self.A.items():
            a.check_guards(name)
        assert np.array_equal(self.A["grad"].bits(), self.A["grad"].before), "the gradients changed"
