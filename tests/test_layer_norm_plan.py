"""How layer norm's forward cuts a call: host arithmetic, compiled here with the
host's own compiler (tests/pins/layer_norm_plan.cpp)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_cuts_of_every_width_fit_an_sm(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not found")
    exe = str(tmp_path / "layer_norm_plan")
    subprocess.run([gxx, "-std=c++17", "-O2", "-Wall", "-Wextra", "-Werror", "-Wno-unused-function", "-I",
                    os.path.join(ROOT, "window_gather_swin_gb300", "csrc"),
                    os.path.join(ROOT, "tests", "pins", "layer_norm_plan.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout
    assert r.stdout.startswith("cuts ")
