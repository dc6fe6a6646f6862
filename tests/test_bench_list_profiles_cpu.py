"""The summaries of a profile of the step over a list of tensors: which code
they are of."""

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
