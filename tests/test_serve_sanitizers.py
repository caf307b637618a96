"""Address and undefined-behaviour sanitizer run of the decoding operators' host
code (argument checks, sizes), with the kernel
launchers replaced by checking stand-ins."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SAN = os.path.join(ROOT, "tests", "sanitize")


def test_serve_abi_host_under_asan_ubsan(tmp_path):
    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(hipcc):
        pytest.skip("hipcc not available")
    exe = str(tmp_path / "serve_san")
    cmd = [hipcc, "--offload-arch=gfx950", "-std=c++17", "-g", "-O1",
           "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-sanitize-recover=all",
           "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
           "-o", exe, os.path.join(SAN, "serve_driver.cpp"), os.path.join(SAN, "serve_stubs.cpp"),
           os.path.join(ROOT, "fp4_quantization_amd", "csrc", "ufp4_serve_api.hip"),
           os.path.join(ROOT, "fp4_quantization_amd", "csrc", "ufp4_host.hip")]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300,
                       env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1",
                                UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1"))
    assert r.returncode == 0 and "passed" in r.stdout, r.stdout + r.stderr
