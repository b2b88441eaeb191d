"""The block operators' host code (csrc/api_block.cpp) under AddressSanitizer and
UndefinedBehaviorSanitizer, driven on the CPU by tests/host/block_driver.cpp with
the HIP runtime and the launchers stubbed: argument rules, workspace rules, the
choice of the kernel family and the mapping of failures.  No GPU is involved."""
import os
import subprocess

import pytest

from tests.test_host_sanitized import CLANG, CSRC, ROOT, SAN, _hipcc

DRIVER = os.path.join(ROOT, "tests", "host", "block_driver.cpp")


def test_block_host_code_under_asan_ubsan(tmp_path):
    if not os.path.exists(_hipcc()) or not os.path.exists(CLANG):
        pytest.skip("ROCm compilers not available")
    objs = []
    for src in (os.path.join(CSRC, "api_block.cpp"), DRIVER):
        obj = str(tmp_path / (os.path.basename(src) + ".o"))
        cmd = [_hipcc(), "-x", "hip", "--cuda-host-only", "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer"] + SAN + [
            "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-c", src, "-o", obj]
        res = subprocess.run(cmd, capture_output=True, text=True)
        assert res.returncode == 0, res.stderr[-3000:]
        objs.append(obj)
    exe = str(tmp_path / "block_driver")
    link = [CLANG, "-fsanitize=address,undefined"] + objs + ["-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib",
                                                            "-o", exe]
    res = subprocess.run(link, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-3000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0", UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    res = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=120)
    assert res.returncode == 0, res.stdout[-3000:] + res.stderr[-3000:]
    assert "all checks passed" in res.stdout
    assert "runtime error" not in res.stderr and "ERROR: AddressSanitizer" not in res.stderr
