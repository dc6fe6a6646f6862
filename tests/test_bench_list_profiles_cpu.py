"""The summaries of a profile of the step over a list of tensors: which code
they are of, and the 8-bit update's bytes however many waves share a unit."""

import os
import shutil

import pytest

import bench
from fsdp_sharded_mixed_zero_amd import synth, zero
from test_bench_cpu import FINAL, NS, _setup_launches, _write_csv

pytestmark = pytest.mark.skipif(not os.path.exists(zero.LIB_PATH),
                                reason="libzero_mi355x.so not built (run __graft_entry__.build())")


def summary(tmp_path, updates, wl, list_bits):
    """The summary of a trace of three steps with these update kernels in each, 2 us a launch."""
    _, trace = _setup_launches(wl)
    t = 1_000_000
    for _ in range(3):
        for name, ns in [("tensors_sqnorm_kernel<unsigned short>(SqArgs)", 1000), *((u, 2000) for u in updates)]:
            trace.append({"Kernel_Name": f"void {NS}{name}", "Start_Timestamp": t, "End_Timestamp": t + ns})
            t += ns + 500
        trace.append({"Kernel_Name": FINAL, "Start_Timestamp": t, "End_Timestamp": t + 100})
        t += 500
    _write_csv(str(tmp_path / "prof" / "bench_kernel_trace.csv"),
               ["Kernel_Name", "Start_Timestamp", "End_Timestamp"], trace)
    return bench.stats_summary(str(tmp_path / "prof"), wl, steps=2, warmup=1, list_bits=list_bits)


@pytest.mark.parametrize("changed", ["tensors.hip", "tensors_internal.h", "kernels.hip"])
def test_a_list_profile_names_the_code_of_its_kernels(tmp_path, monkeypatch, changed):
    kind = f"{NS}StepArgs"
    update = f"tensors_adamw_kernel<unsigned short, unsigned short>({kind})"
    here = tmp_path / "csrc"
    shutil.copytree(bench.CSRC, here)
    monkeypatch.setattr(bench, "CSRC", str(here))
    monkeypatch.setattr(bench, "KERNEL_SOURCE", str(here / "kernels.hip"))
    wl = synth.WORKLOADS["tiny"]
    before, flat = summary(tmp_path, [update], wl, 32), bench.source_hash()
    line = [x for x in before.splitlines() if "sha256" in x]
    assert len(line) == 1 and all(name in line[0] for name in bench.LIST_SOURCES)
    path = here / changed
    text = path.read_text(encoding="utf-8")
    path.write_text(text + "\n// a comment\n", encoding="utf-8")
    assert line[0] in summary(tmp_path, [update], wl, 32)
    path.write_text(text + "\nint one_more;\n", encoding="utf-8")
    assert line[0] not in summary(tmp_path, [update], wl, 32)
    assert (bench.source_hash() == flat) == (changed != "kernels.hip")


@pytest.mark.parametrize("waves", [(1,), (2,), (4,), (1, 4)])
def test_the_8_bit_update_has_its_bytes(tmp_path, waves):
    wl = synth.WORKLOADS["tiny"]
    md = summary(tmp_path, [f"tensors_adamw8_kernel<unsigned short, unsigned short, {w}>({NS}StepArgs)" for w in waves],
                 wl, 8)
    _, _, algo = bench.algorithmic_bytes(wl, list_bits=8)
    want = algo["tensors_adamw8_kernel<unsigned short, unsigned short, 1>"]
    rows = [[c.strip() for c in line.split("|")[1:-1]] for line in md.splitlines() if line.startswith("| tensors_adamw8")]
    assert len(rows) == 1 and all(f" {w}" in rows[0][0] for w in waves)
    assert int(rows[0][1]) == 3 * len(waves) and float(rows[0][2]) == len(waves)
    assert int(rows[0][6]) == int(want / len(waves))
    assert float(rows[0][9]) == pytest.approx(2.0 * len(waves))


def test_a_list_has_no_buckets(tmp_path):
    """The step over a list is not cut into the workload's buckets."""
    wl = synth.WORKLOADS["llama-70b"]
    assert wl.bucket > 0
    md = summary(tmp_path, [f"tensors_adamw_kernel<unsigned short, unsigned short>({NS}StepArgs)"], wl, 32)
    assert "buckets" not in md.splitlines()[0] and "3 steps traced" in md     # the path of the trace has this test's name
