"""Registers that the warpgroups of the large product share, from ptxas's resource report
(no GPU)."""
import ctypes
import os
import shutil
import subprocess

import pytest

from test_kernel_resources import CSRC, ROOT, _find, ptxas_report

pytestmark = pytest.mark.skipif(shutil.which("nvcc") is None, reason="nvcc not available")


@pytest.fixture(scope="module")
def product():
    return ptxas_report("matmul_fp8.cu")


@pytest.fixture(scope="module")
def suffices(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("split") / "libsplit.so")
    subprocess.run(["nvcc", "-O2", "-std=c++17", "-Xcompiler", "-fPIC", "-shared", "-I", CSRC, "-o", out,
                    os.path.join(ROOT, "tests", "c", "register_split.cu")], check=True)
    f = ctypes.CDLL(out).split_suffices
    f.argtypes, f.restype = [ctypes.c_int], ctypes.c_int
    return f


def test_the_split_is_checked_against_what_a_block_is_launched_with(suffices):
    for regs in range(0, 256, 8):
        assert suffices(regs) == (regs * 384 >= 56 * 128 + 224 * 256), regs
    assert suffices(168) and not suffices(160)


@pytest.mark.parametrize("column_scales", [0, 1])
def test_large_product_has_the_registers_that_its_warpgroups_share(product, suffices, column_scales):
    # fewer at launch and the warpgroups that ask for 224 would never get them
    k = _find(product, f"k_matmul_pairILb{column_scales}E")
    assert k["regs"] == 168 and k["spill"] == 0 and suffices(k["regs"])


def test_large_product_is_refused_where_they_are_fewer():
    text = open(os.path.join(CSRC, "matmul_fp8.cu")).read()
    launch = text[text.index("cudaError_t launch_pair("):]
    launch = launch[:launch.index("\n}\n")]
    assert "cudaFuncGetAttributes" in launch and "registers_suffice(" in launch
    assert launch.index("registers_suffice(") < launch.index("launch_kernel(")
