"""The quantizer's asynchronous copies of bf16 rows off 16-byte boundaries, walked on
the CPU: a 16-byte copy starts on a 16-byte boundary inside its row, also where nothing
of the granule is left (then there is no copy)."""
import ctypes
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "shared_memory_tiled_gb300", "csrc")

pytestmark = pytest.mark.skipif(shutil.which("nvcc") is None, reason="nvcc not available")


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("granule") / "libgranule.so")
    subprocess.run(["nvcc", "-O2", "-std=c++17", "-Xcompiler", "-fPIC", "-shared", "-I", CSRC, "-o", out,
                    os.path.join(ROOT, "tests", "c", "granule.cu")], check=True)
    f = ctypes.CDLL(out).granule_faults
    f.argtypes = [ctypes.c_ulonglong] + [ctypes.c_longlong] * 3 + [ctypes.POINTER(ctypes.c_longlong)]
    f.restype = ctypes.c_longlong
    return f


@pytest.mark.parametrize("off", range(8))
def test_copies_start_on_boundaries_inside_their_rows(walk, off):
    for cols in [1, 7, 8, 9, 100, 121, 127, 128, 129, 135, 136, 255, 256, 257, 300, 1000, 7919]:
        for ld in (cols, cols + 1, cols + 5):
            base, rows = (1 << 20) + 2 * off, 9
            taken = ctypes.c_longlong(0)
            assert walk(base, rows, cols, ld, ctypes.byref(taken)) == 0, (cols, ld)
            # A tile's first 16 granules end where the next tile's begin: of a row they miss
            # less than one at its start, and less than the last tile's 17th at its end.
            assert 2 * rows * cols - rows * 32 < taken.value <= 2 * rows * cols
