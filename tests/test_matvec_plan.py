"""The choice of a product's launch on the host: what each kernel takes for granted
holds for every size, sums over no values among them."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_every_choice_fits_its_kernel(tmp_path):
    gxx = shutil.which("g++")
    if not gxx:
        pytest.skip("g++ not available")
    exe = str(tmp_path / "plan")
    r = subprocess.run([gxx, "-std=c++17", "-g", "-O1", "-Wall", "-o", exe,
                        os.path.join(ROOT, "tests", "sanitize", "matvec_plan_driver.cpp")], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "passed" in r.stdout, r.stdout + r.stderr
