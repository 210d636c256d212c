"""How embedding_bwd cuts a call: host arithmetic, compiled here with the host's own
compiler (tests/pins/embedding_plan.cpp)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_cuts_of_many_sizes_on_few_and_many_sms(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not found")
    exe = str(tmp_path / "embedding_plan")
    subprocess.run([gxx, "-std=c++17", "-O2", "-Wall", "-Wextra", "-Werror", "-I",
                    os.path.join(ROOT, "window_gather_swin_gb300", "csrc"),
                    os.path.join(ROOT, "tests", "pins", "embedding_plan.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout
    assert r.stdout.startswith("plans ")
