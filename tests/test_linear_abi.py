"""The linear layer's entry points on the host: every argument error comes back
before any CUDA call (no GPU needed; the addresses are never dereferenced)."""
from __future__ import annotations

import ctypes

import pytest

from shared_memory_tiled_gb300 import binding as B
from shared_memory_tiled_gb300 import build as build_mod

S = B.Status
AT = [0x7F0000000000 + i * 0x10000000000 for i in range(10)]  # far apart


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build_mod.build()
    B.load()


def quantize(**kw):
    a = B.QuantizeArgs(x=AT[0], q=AT[1], scale=AT[2], qt=AT[3], scale_t=AT[4], x_dtype=B.DType.BF16,
                       q_dtype=B.DType.E4M3, block_rows=1, rows=300, cols=500, ld_x=500, ld_q=512,
                       ld_scale=300, ld_qt=304, ld_scale_t=500)
    for k, v in kw.items():
        setattr(a, k, v)
    return B.tr_quantize_fp8(a)


def test_quantize_refusals():
    assert B.tr_quantize_fp8(None) == S.ERR_NULL
    for bad in (dict(reserved=1), dict(x_dtype=B.DType.E4M3), dict(x_dtype=9), dict(q_dtype=B.DType.F32),
                dict(q_dtype=-1), dict(block_rows=0), dict(block_rows=64)):
        assert quantize(**bad) == S.ERR_UNSUPPORTED, bad
    assert quantize(rows=-1) == S.ERR_BAD_DIM and quantize(cols=-5) == S.ERR_BAD_DIM
    for name in ("x", "q", "scale", "scale_t"):
        assert quantize(**{name: 0}) == S.ERR_NULL, name
    for bad in (dict(ld_x=499), dict(ld_q=496), dict(ld_scale=299), dict(ld_qt=288), dict(ld_scale_t=499)):
        assert quantize(**bad) == S.ERR_BAD_LD, bad
    for bad in (dict(x=AT[0] + 1), dict(q=AT[1] + 8), dict(qt=AT[3] + 1), dict(scale=AT[2] + 2),
                dict(scale_t=AT[4] + 1), dict(ld_q=520), dict(ld_qt=312)):
        assert quantize(**bad) == S.ERR_UNSUPPORTED, bad
    assert "multiple of 16" in B.tr_last_error()
    # outputs over the input, over one another, and over the input's last bytes
    assert quantize(q=AT[0]) == S.ERR_OVERLAP
    assert quantize(qt=AT[1] + 299 * 512) == S.ERR_OVERLAP
    assert quantize(scale=AT[2], scale_t=AT[2] + 16) == S.ERR_OVERLAP
    assert quantize(scale=AT[0] + 2 * (299 * 500 + 498)) == S.ERR_OVERLAP
    assert quantize(rows=1 << 40, ld_x=1 << 40, ld_scale=1 << 40, cols=1 << 30) == S.ERR_BAD_DIM
    # nothing to do, whatever the pointers
    assert quantize(rows=0, x=0, q=0, scale=0, scale_t=0) == S.OK
    assert quantize(cols=0, x=0, q=0) == S.OK


def matmul(**kw):
    a = B.MatmulFp8Args(a=AT[0], scale_a=AT[1], b=AT[2], scale_b=AT[3], out=AT[4], a_dtype=B.DType.E4M3,
                        b_dtype=B.DType.E5M2, out_dtype=B.DType.F32, a_block_rows=1, b_block_rows=128,
                        accumulate=0, m=200, n=300, k=500, lda=512, ldb=512, ld_out=300, ld_scale_a=200,
                        ld_scale_b=3)
    for k, v in kw.items():
        setattr(a, k, v)
    return B.tr_matmul_fp8(a)


def test_matmul_refusals():
    assert B.tr_matmul_fp8(None) == S.ERR_NULL
    for bad in (dict(a_dtype=B.DType.BF16), dict(b_dtype=7), dict(out_dtype=B.DType.E4M3), dict(a_block_rows=2),
                dict(b_block_rows=0), dict(accumulate=2), dict(accumulate=-1), dict(m=1 << 31), dict(k=1 << 31)):
        assert matmul(**bad) == S.ERR_UNSUPPORTED, bad
    for name in "mnk":
        assert matmul(**{name: -1}) == S.ERR_BAD_DIM
    for name in ("a", "b", "scale_a", "scale_b", "out"):
        assert matmul(**{name: 0}) == S.ERR_NULL, name
    for bad in (dict(lda=496), dict(ldb=496), dict(ld_out=299), dict(ld_scale_a=199), dict(ld_scale_b=2)):
        assert matmul(**bad) == S.ERR_BAD_LD, bad
    for bad in (dict(a=AT[0] + 8), dict(b=AT[2] + 1), dict(scale_a=AT[1] + 1), dict(out=AT[4] + 2),
                dict(lda=504), dict(ldb=520)):
        assert matmul(**bad) == S.ERR_UNSUPPORTED, bad
    assert matmul(out=AT[0]) == S.ERR_OVERLAP
    assert matmul(out=AT[3] + 4 * (3 * 3 + 2)) == S.ERR_OVERLAP
    assert matmul(m=0, a=0, out=0) == S.OK and matmul(n=0, b=0, out=0) == S.OK
    # no contraction and an old value to keep: nothing to do
    assert matmul(k=0, a=0, b=0, scale_a=0, scale_b=0, accumulate=1) == S.OK


def layernorm(**kw):
    a = B.LayernormArgs(x=AT[0], gamma=AT[1], beta=AT[2], y=AT[3], mean=AT[4], rstd=AT[5], x_dtype=B.DType.BF16,
                        w_dtype=B.DType.F32, rows=20, cols=30, ld_x=30, ld_y=32, eps=1e-5)
    for k, v in kw.items():
        setattr(a, k, v)
    return B.tr_layernorm(a)


def test_layernorm_refusals():
    assert B.tr_layernorm(None) == S.ERR_NULL
    for bad in (dict(x_dtype=2), dict(w_dtype=3), dict(reserved=1)):
        assert layernorm(**bad) == S.ERR_UNSUPPORTED, bad
    for bad in (dict(rows=-1), dict(cols=-1), dict(eps=-1e-9), dict(eps=float("nan")), dict(eps=float("inf"))):
        assert layernorm(**bad) == S.ERR_BAD_DIM, bad
    for name in ("x", "gamma", "y"):
        assert layernorm(**{name: 0}) == S.ERR_NULL, name
    assert layernorm(ld_x=29) == S.ERR_BAD_LD and layernorm(ld_y=29) == S.ERR_BAD_LD
    for bad in (dict(x=AT[0] + 1), dict(gamma=AT[1] + 2), dict(beta=AT[2] + 1), dict(y=AT[3] + 1), dict(mean=AT[4] + 2),
                dict(rstd=AT[5] + 3)):
        assert layernorm(**bad) == S.ERR_UNSUPPORTED, bad
    for bad in (dict(y=AT[0]), dict(y=AT[1] + 116), dict(mean=AT[0]), dict(mean=AT[4], rstd=AT[4] + 4),
                dict(mean=AT[3])):
        assert layernorm(**bad) == S.ERR_OVERLAP, bad
    assert layernorm(rows=0, x=0, y=0) == S.OK and layernorm(cols=0, x=0, gamma=0, y=0) == S.OK


def layernorm_backward(**kw):
    a = B.LayernormBackwardArgs(dy=AT[0], x=AT[1], gamma=AT[2], mean=AT[3], rstd=AT[4], dx=AT[5], dgamma=AT[6],
                                dbeta=AT[7], workspace=AT[8], workspace_bytes=1 << 20, x_dtype=B.DType.BF16,
                                w_dtype=B.DType.F32, rows=20, cols=30, ld_dy=30, ld_x=30, ld_dx=30)
    for k, v in kw.items():
        setattr(a, k, v)
    return B.tr_layernorm_backward(a)


def test_layernorm_backward_refusals():
    assert B.tr_layernorm_backward(None) == S.ERR_NULL
    for bad in (dict(x_dtype=2), dict(w_dtype=9)):
        assert layernorm_backward(**bad) == S.ERR_UNSUPPORTED, bad
    assert layernorm_backward(rows=-1) == S.ERR_BAD_DIM and layernorm_backward(cols=-1) == S.ERR_BAD_DIM
    for name in ("dy", "x", "gamma", "mean", "rstd", "dx", "dgamma", "workspace"):
        assert layernorm_backward(**{name: 0}) == S.ERR_NULL, name
    for bad in (dict(ld_dy=29), dict(ld_x=29), dict(ld_dx=29)):
        assert layernorm_backward(**bad) == S.ERR_BAD_LD, bad
    need = B.tr_layernorm_backward_workspace(20, 30)
    for bad in (dict(workspace_bytes=need - 1), dict(workspace=AT[8] + 8), dict(dgamma=AT[6] + 2), dict(dx=AT[5] + 1),
                dict(mean=AT[3] + 2)):
        assert layernorm_backward(**bad) == S.ERR_UNSUPPORTED, bad
    for bad in (dict(dx=AT[0]), dict(dx=AT[1]), dict(dgamma=AT[2]), dict(dbeta=AT[6] + 116), dict(workspace=AT[5]),
                dict(workspace=AT[3])):
        assert layernorm_backward(**bad) == S.ERR_OVERLAP, bad
    assert layernorm_backward(cols=0, dgamma=0) == S.OK


def test_layernorm_backward_workspace():
    f = B.tr_layernorm_backward_workspace
    assert f(0, 100) == 0 and f(100, 0) == 0
    assert f(-1, 4) == -1 and f(4, -1) == -1 and f(1 << 40, 1 << 60) == -1
    for rows, cols in [(1, 1), (20, 30), (5000, 1024), (5000, 2000), (100000, 8192), (7, 70001)]:
        n = f(rows, cols)
        assert n % (8 * cols) == 0 and 0 < n // (8 * cols) <= rows  # two fp32 sums for each part and column


def test_argument_structs_match_the_header():
    """Field order and sizes, as a C compiler sees them."""
    import os
    import re
    import shutil
    import subprocess
    import tempfile
    if shutil.which("gcc") is None:
        pytest.skip("gcc not available")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    names = {"tr_quantize_args": B.QuantizeArgs, "tr_matmul_fp8_args": B.MatmulFp8Args,
             "tr_layernorm_args": B.LayernormArgs, "tr_layernorm_backward_args": B.LayernormBackwardArgs}
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "transpose.h"', "int main(void) {"]
    for c, py in names.items():
        lines.append(f'printf("{c} %zu\\n", sizeof({c}));')
        lines += [f'printf("{c}.{f} %zu\\n", offsetof({c}, {f}));' for f, _ in py._fields_]
    with tempfile.TemporaryDirectory() as d:
        src, exe = os.path.join(d, "s.c"), os.path.join(d, "s")
        open(src, "w").write("\n".join(lines + ["return 0; }"]))
        subprocess.run(["gcc", "-std=c99", "-I", os.path.join(root, "include"), src, "-o", exe], check=True)
        out = subprocess.run([exe], capture_output=True, text=True, check=True).stdout
    got = dict(line.rsplit(" ", 1) for line in out.split("\n") if line)
    for c, py in names.items():
        assert int(got[c]) == ctypes.sizeof(py)
        for f, _ in py._fields_:
            assert int(got[f"{c}.{f}"]) == getattr(py, f).offset, (c, f)
        assert len(re.findall(rf"^{c}\.", out, flags=re.M)) == len(py._fields_)


def test_conveniences_refuse_what_they_cannot_take():
    import torch
    x = torch.zeros(4, 8)
    for call in (lambda: B.quantize_fp8(x), lambda: B.layernorm(x, x[0]),
                 lambda: B.layernorm_backward(x, x, x[0], x[:, 0], x[:, 0]), lambda: B.matmul_fp8(x, x, x, x),
                 lambda: B.quantize_fp8(x, stream=0)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
