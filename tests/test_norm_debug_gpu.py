"""Root-mean-square norm and the adapters through the bounds-checked build: every global load and store that their
kernels make themselves is checked against its operand first (tiles that TMA moves are clipped to their tensor
maps), results are those of the release build, and nothing is refused."""
from __future__ import annotations

import pytest

from shared_memory_tiled_gb300 import binding as B
from test_adapters_gpu import problem
from test_linear_debug_gpu import both, dlib, view  # noqa: F401

pytestmark = pytest.mark.gpu

SHAPES = [(1, 1, 1, 0), (3, 128, 128, 0), (300, 520, 520, 0), (300, 520, 521, 0), (129, 1000, 1003, 5), (260, 8, 9, 1), (5, 16400, 16400, 0),
          (3, 8192, 8192, 0), (700, 2048, 2048, 0)]


@pytest.mark.parametrize("kind", ["bfloat16", "float32"])
def test_rmsnorm(monkeypatch, dlib, kind):  # noqa: F811
    import torch
    for rows, cols, pitch, off in SHAPES:
        x = view(rows, cols, pitch, off, getattr(torch, kind))
        gamma = torch.rand(cols, device="cuda")
        for res in (None, x):
            both(monkeypatch, dlib, lambda: B.rmsnorm(x, gamma, res))
            both(monkeypatch, dlib, lambda: B.rmsnorm_fp8(x, gamma, res, transposed=True))
            rstd = B.rmsnorm(x, gamma, res)[2]
            both(monkeypatch, dlib, lambda: B.rmsnorm_backward(x, x, gamma, rstd, dresidual=res))


@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_adapters(monkeypatch, dlib, out):  # noqa: F811
    import torch
    for tokens, count, k, n, rank in [(1, 2, 40, 30, 8), (30, 3, 100, 77, 5), (150, 3, 264, 140, 16), (300, 2, 520, 256, 64), (2100, 40, 72, 136, 100)]:
        p, w = problem(tokens, count, k, n, rank, 1, out)
        index = torch.from_numpy(w[4]).cuda()

        def call():
            plan = B.adapter_plan(index, count)
            return [B.adapters(p["x"], p["a"], p["b"], plan, scale=p["scale"], base=base, out_dtype=p["base"].dtype) for base in (p["base"], None)]
        both(monkeypatch, dlib, call)
