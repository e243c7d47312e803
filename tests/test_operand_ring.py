"""The product's ring of operand stages, walked on the CPU: when the warp that loads has
left it, no load and no commit is in flight to shared memory that the block gives up,
whether every block of the contraction was computed or the instructions gave up
on the way."""
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
    out = str(tmp_path_factory.mktemp("ring") / "libring.so")
    subprocess.run(["nvcc", "-O2", "-std=c++17", "-Xcompiler", "-fPIC", "-shared", "-I", CSRC, "-o", out,
                    os.path.join(ROOT, "tests", "c", "operand_ring.cu")], check=True)
    f = ctypes.CDLL(out).ring_leftovers
    f.argtypes = [ctypes.c_int, ctypes.c_longlong, ctypes.c_longlong, ctypes.c_uint, ctypes.POINTER(ctypes.c_int)]
    f.restype = ctypes.c_longlong

    def call(stages, blocks, gives_up_at, seed):
        ok = ctypes.c_int(-1)
        return f(stages, blocks, gives_up_at, seed, ctypes.byref(ok)), bool(ok.value)
    return call


@pytest.mark.parametrize("stages", [2, 3, 4, 5])
def test_nothing_is_in_flight_after_a_whole_contraction(walk, stages):
    for blocks in list(range(0, 3 * stages + 2)) + [64, 129]:
        for seed in range(30):
            assert walk(stages, blocks, blocks, seed) == (0, True), (blocks, seed)


@pytest.mark.parametrize("stages", [2, 3, 4, 5])
def test_nothing_is_in_flight_after_the_instructions_gave_up(walk, stages):
    for blocks in range(1, 3 * stages + 2):
        for gives_up_at in range(blocks):
            for seed in range(20):
                assert walk(stages, blocks, gives_up_at, seed) == (0, False), (blocks, gives_up_at, seed)
