"""What wgs_check_error makes of the device's error words: a bad index and a
kernel that gave up waiting for its own copies are each reported, one check
after the other when both were seen.

The library's own objects are linked to the shared CUDA runtime, of which
tests/pins/error_words.c replaces the calls that would reach a GPU.
"""
import glob
import os
import shutil
import subprocess
import sys

import pytest

from window_gather_swin_gb300 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = """
import ctypes, sys
fake = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
check = ctypes.CDLL(sys.argv[2]).wgs_check_error
check.argtypes = [ctypes.c_void_p]
OK, LAUNCH, INDEX = 0, 7, 8
ROWS, MASK, BUCKET, NORM = range(4)

def after(**words):
    for name, value in words.items():
        fake.fake_set_word(globals()[name], value)
    return [check(None) for _ in range(3)]

assert after() == [OK, OK, OK]                 # and names the words, in this order
assert after(ROWS=1) == [INDEX, OK, OK]
assert after(MASK=1) == [INDEX, OK, OK]
assert after(BUCKET=1) == [INDEX, OK, OK]
assert after(BUCKET=2) == [LAUNCH, OK, OK]
assert after(NORM=1) == [LAUNCH, OK, OK]
assert after(ROWS=1, NORM=1) == [LAUNCH, INDEX, OK]
assert after(MASK=1, BUCKET=2) == [LAUNCH, INDEX, OK]
assert after(BUCKET=3) == [LAUNCH, INDEX, OK]
assert after(ROWS=1, MASK=1, BUCKET=3, NORM=1) == [LAUNCH, INDEX, OK]
"""


def test_both_kinds_of_error_are_reported(tmp_path):
    gcc, nvcc = shutil.which("gcc"), build.nvcc()
    if gcc is None:
        pytest.skip("gcc not found")
    build.build()
    objects = sorted(glob.glob(os.path.join(build.LIB_DIR, "obj", "*.o")))
    if not objects:
        build.build(force=True)
        objects = sorted(glob.glob(os.path.join(build.LIB_DIR, "obj", "*.o")))
    lib, fake = str(tmp_path / "libwgs_shared_rt.so"), str(tmp_path / "libfake.so")
    subprocess.run([nvcc, "-shared", "-o", lib] + objects + build.ARCH + ["-cudart", "shared"], check=True,
                   capture_output=True, timeout=120)
    subprocess.run([gcc, "-shared", "-fPIC", "-Wall", "-Werror", "-o", fake,
                    os.path.join(ROOT, "tests", "pins", "error_words.c")], check=True, timeout=60)
    libs = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "lib64")
    env = {**os.environ, "LD_PRELOAD": fake,
           "LD_LIBRARY_PATH": libs + os.pathsep + os.environ.get("LD_LIBRARY_PATH", "")}
    r = subprocess.run([sys.executable, "-c", CHILD, fake, lib], env=env, capture_output=True, text=True,
                       timeout=120)
    assert r.returncode == 0, r.stderr[-1500:]
