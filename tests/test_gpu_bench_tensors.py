"""bench.py --per-tensor on the GPU, on the tiny workload: the benchmark's JSON
line with the list's kernels and bytes, for moments in 32 and in 8 bits."""

import json
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("bits", [32, 8])
def test_bench_per_tensor(bits):
    cmd = [sys.executable, os.path.join(ROOT, "bench.py"), "--workload", "tiny", "--steps", "5", "--warmup", "2",
           "--per-tensor", "--state-bits", str(bits), "--no-cpu-baseline", "--no-copy-ceiling"]
    print("\n[bench tiny]", " ".join(cmd[1:]), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=100, cwd=ROOT)
    assert r.returncode == 0, r.stderr[-2000:]
    lines = [line for line in r.stdout.splitlines() if line.strip()]
    assert len(lines) == 1
    d = json.loads(lines[0])
    assert d["steps"] == 5 and d["warmup"] == 2 and d["n_gpus"] == 1 and d["value"] > 0
    assert d["config"]["state"] == f"tensor by tensor, moments in {bits} bits"
    S = d["config"]["shard_params"]                 # no padding in this shard
    assert set(d["kernels"]) == {"sqnorm", "adamw"}
    assert d["kernels"]["sqnorm"]["algorithmic_bytes"] == 2 * S
    update = d["kernels"]["adamw"]["algorithmic_bytes"]
    assert update == 28 * S if bits == 32 else 16 * S < update < 17 * S
    assert d["roofline"]["algorithmic_bytes_per_launch"] == update
