"""The host code of the token-table and norm calls (their checks) under
AddressSanitizer and UndefinedBehaviorSanitizer, and built with GCC: a host-only
build with the launches stubbed runs the host tests in a child process. Any report
aborts the child."""

import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "fsdp_sharded_mixed_zero_amd", "csrc")
CLANG = "/opt/rocm/lib/llvm/bin/clang++"
SANITIZE = os.path.join(ROOT, "tests", "sanitize")


def build_and_run(cxx, flags, lib, env):
    build = [cxx, "-shared", "-fPIC", *flags, "-std=c++17", "-Wall", "-Werror", "-fno-math-errno", "-ffp-contract=off",
             "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-I", "/opt/rocm/include",
             *[os.path.join(CSRC, f) for f in ("layout.cpp", "offload.cpp", "tensors.cpp", "layers.cpp")],
             *[os.path.join(SANITIZE, f) for f in ("device_stubs.cpp", "tensor_stubs.cpp", "layer_stubs.cpp")], "-pthread", "-o", lib]
    r = subprocess.run(build, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider", "-m", "not gpu",
                        "tests/test_layers_abi_cpu.py"], cwd=ROOT, env=dict(os.environ, ZERO_MI355X_LIB=lib, **env),
                       capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, (r.stdout[-3000:], r.stderr[-3000:])
    assert " passed" in r.stdout


def test_host_code_under_sanitizers(tmp_path):
    if not os.path.exists(CLANG):
        pytest.skip("ROCm clang++ not found")
    runtime = subprocess.run([CLANG, "-print-file-name=libclang_rt.asan-x86_64.so"], capture_output=True,
                             text=True).stdout.strip()
    if not os.path.isabs(runtime) or not os.path.exists(runtime):
        pytest.skip("sanitizer runtime not found")
    build_and_run(CLANG, ["-O1", "-g", "-fno-omit-frame-pointer", "-fsanitize=address,undefined",
                          "-fno-sanitize-recover=undefined", "-shared-libsan"],
                  str(tmp_path / "libzero_host_sanitized.so"),
                  dict(LD_PRELOAD=runtime, ASAN_OPTIONS="detect_leaks=0:alloc_dealloc_mismatch=0:abort_on_error=1",
                       UBSAN_OPTIONS="print_stacktrace=1"))


def test_host_code_built_with_gcc(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("g++ not found")
    build_and_run("g++", ["-O3"], str(tmp_path / "libzero_host_gcc.so"), {})
