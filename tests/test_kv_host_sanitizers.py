"""The host code of the entry points around a paged FP4 cache (validation, launch plans) under AddressSanitizer and
UndefinedBehaviorSanitizer (CPU only): tests/sanitize/kv_abi_driver.cpp calls them with null, misaligned and aliasing
pointers and sizes from -1 to INT64_MAX."""
import os
import subprocess

import pytest

from nvfp4_weight_only_amd import build as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_kv_abi_validation_under_asan_ubsan(tmp_path):
    rocm = os.path.dirname(os.path.dirname(os.path.realpath(B.hipcc())))
    clang = os.path.join(rocm, "lib", "llvm", "bin", "clang++")
    if not os.path.exists(clang):
        pytest.skip("ROCm clang++ not found")
    lib = B.build_host_sanitized(str(tmp_path))
    exe = str(tmp_path / "kv_abi_driver")
    subprocess.run([clang, "-O1", "-g", "-std=c++17", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
                    "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(rocm, "include"), "-I", os.path.join(ROOT, "include"),
                    os.path.join(ROOT, "tests", "sanitize", "kv_abi_driver.cpp"), lib, "-o", exe,
                    "-L" + os.path.join(rocm, "lib"), "-lamdhip64", "-Wl,-rpath," + os.path.join(rocm, "lib"),
                    "-Wl,-rpath," + str(tmp_path)], check=True)
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1", UBSAN_OPTIONS="print_stacktrace=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=600)
    out = r.stdout + r.stderr
    assert r.returncode == 0, out[-4000:]
    assert "runtime error" not in out and "AddressSanitizer" not in out, out[-4000:]
    assert "calls" in out or "skipped" in out, out[-2000:]
