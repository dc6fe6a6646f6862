"""The benchmark's list-of-tensors mode on the host: its bytes per kernel and
the flag combinations it refuses."""

import os
import subprocess
import sys

import pytest

import bench
from fsdp_sharded_mixed_zero_amd import synth, zero

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("name", ["tiny", "gpt2-1.5b", "gpt-7.5b", "llama-7b"])
def test_algorithmic_bytes_of_a_list(name):
    wl = synth.WORKLOADS[name]
    lay = zero.zero_layout(wl.sizes, wl.n_d, wl.rank, wl.align)
    lens = [s[3] for s in lay.segments]
    S, real, b32 = bench.algorithmic_bytes(wl, list_bits=32)
    assert (S, real) == (lay.info["shard"], sum(lens))
    # gradient 2, parameter 2, master, m and v read and written
    assert b32 == {"tensors_sqnorm_kernel<unsigned short>": 2 * real,
                   "tensors_adamw_kernel<unsigned short, unsigned short>": (2 + 2 + 3 * 8) * real}
    # both moments a byte, and a scale of 4 bytes per 256 elements of a tensor, read and written
    blocks = sum((n + 255) // 256 for n in lens)
    _, _, b8 = bench.algorithmic_bytes(wl, list_bits=8)
    assert b8["tensors_adamw8_kernel<unsigned short, unsigned short, 1>"] == (2 + 2 + 8 + 4) * real + 16 * blocks


@pytest.mark.parametrize("flags", [["--per-tensor", "--flat"], ["--per-tensor", "--accum", "2"],
                                   ["--per-tensor", "--offload"], ["--per-tensor", "--state-arrays"],
                                   ["--state-bits", "8"]])
def test_refused_combinations(flags):
    r = subprocess.run([sys.executable, os.path.join(ROOT, "bench.py"), *flags], capture_output=True, text=True,
                       timeout=120, cwd=ROOT)
    assert r.returncode != 0 and "--per-tensor" in r.stderr and not r.stdout.strip()
