"""The linear layer's operators through the bounds-checked build: every global load
and store that their kernels make themselves is checked against its operand first
(tiles that TMA moves are clipped to their tensor maps), results are right, and
nothing is refused."""
from __future__ import annotations

import ctypes

import pytest

from shared_memory_tiled_gb300 import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dlib():
    from shared_memory_tiled_gb300 import build
    return B.open_library(build.build(debug=True))


def refused(lib):
    rep = B.BoundsReport()
    assert lib.tr_debug_bounds(ctypes.byref(rep)) == B.Status.OK
    return rep.refused, hex(rep.first_address), rep.first_bytes, rep.first_store


def both(monkeypatch, dlib, call):
    """The release build's answer and the bounds-checked one's."""
    import torch
    want = call()
    refused(dlib)
    with monkeypatch.context() as m:
        m.setattr(B, "_lib", dlib)
        got = call()
        torch.cuda.synchronize()
    assert refused(dlib)[0] == 0, refused(dlib)
    for a, b in zip(got, want):
        if a is not None:
            assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def view(rows, cols, pitch, off, dtype):
    import torch
    g = torch.Generator(device="cuda").manual_seed(rows * 7 + cols)
    buf = torch.randn(off + rows * pitch, device="cuda", generator=g).to(dtype)
    return buf[off:].view(rows, pitch)[:, :cols]


@pytest.mark.parametrize("kind", ["bfloat16", "float32"])
def test_quantize(monkeypatch, dlib, kind):
    import torch
    dt = getattr(torch, kind)
    for rows, cols, pitch, off in [(1, 1, 1, 0), (300, 520, 520, 0), (300, 520, 521, 0), (129, 1000, 1003, 5), (260, 8, 9, 1)]:
        x = view(rows, cols, pitch, off, dt)
        for block in (1, 128):
            both(monkeypatch, dlib, lambda: B.quantize_fp8(x, block_rows=block, transposed=True))


def test_product(monkeypatch, dlib):
    import torch
    for m, n, k in [(1, 300, 1000), (40, 129, 333), (200, 333, 2048), (777, 513, 1111), (2435, 2311, 300)]:
        for ab, bb in [(1, 128), (1, 1), (128, 128)]:
            a = B.quantize_fp8(view(m, k, k, 0, torch.float32), block_rows=ab)
            b = B.quantize_fp8(view(n, k, k, 0, torch.float32), block_rows=bb)
            both(monkeypatch, dlib, lambda: (B.matmul_fp8(*a, *b),))
            out = torch.zeros(m, n + 3, device="cuda")[:, :n]
            both(monkeypatch, dlib, lambda: (B.matmul_fp8(*a, *b, out=out),))


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_layernorm(monkeypatch, dlib, kind):
    """Against the 64-bit forms: the two builds may contract a multiplication and an
    addition differently."""
    from test_linear_gpu import check_layernorm, check_layernorm_backward
    refused(dlib)
    monkeypatch.setattr(B, "_lib", dlib)
    for rows, cols, pitch, off in [(1, 1, 1, 0), (3, 96, 96, 0), (5, 1000, 1001, 3), (6000, 300, 301, 1),
                                   (5000, 1024, 1024, 0), (7, 20001, 20001, 0), (40, 9000, 9000, 0)]:
        check_layernorm(rows, cols, kind, "f32", rows, pitch=pitch, off=off)
        check_layernorm_backward(rows, cols, kind, "f32", rows, pitch=pitch, off=off)
        assert refused(dlib)[0] == 0, (rows, cols, refused(dlib))
