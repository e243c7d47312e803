"""Infinite and very large values in the adapters' second product, by what their definition gives."""
from __future__ import annotations

import numpy as np
import pytest

from shared_memory_tiled_gb300 import binding as B
from test_adapters_gpu import _lib, held, up8  # noqa: F401
from test_linear_gpu import torch_types

pytestmark = pytest.mark.gpu

INF = float("inf")


def problem(tokens, rank, n, out, seed):
    """Integers, so that every inner value is exact and many are exact in bf16 or zero."""
    import torch
    rng = np.random.default_rng(seed)
    x, wx = held(rng.integers(-2, 3, (tokens, 72)), 72)
    a, wa = held(rng.integers(-2, 3, (2, rank, 72)), 72)
    b, wb = held(rng.integers(-3, 4, (2, n, rank)), up8(rank))
    base = torch.from_numpy(rng.integers(-9, 10, (tokens, n))).to(torch_types(out)).cuda()
    index = torch.from_numpy((np.arange(tokens) % 3 - 1).astype(np.int32)).cuda()
    return x, a, b, base, index


def want(x, a, b, base, index, scale):
    import torch
    out = base.double()
    for g in range(2):
        at = index == g
        v = scale[g].double() * (x[at].double() @ a[g].double().t())
        out[at] += (v[:, None, :] * b[g].double()[None]).sum(2)   # zero times infinity is NaN, unlike infinities are
    return out.to(base.dtype)


# both kernels, and both in one call; outputs on and off 16-byte boundaries; each width of the inner values
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("tokens,rank,n", [(5, 5, 40), (30, 32, 41), (24, 64, 40), (31, 128, 33), (90, 16, 40), (600, 24, 41), (700, 16, 136), (600, 64, 40),
                                           (600, 100, 41), (2100, 8, 40), (2100, 33, 136)])
def test_infinite_b(tokens, rank, n, out):
    import torch
    x, a, b, base, index = problem(tokens, rank, n, out, tokens + rank)
    scale = torch.tensor([1.0, 0.7], device="cuda")
    plan = B.adapter_plan(index, 2)
    clean = B.adapters(x, a, b, plan, scale=scale, base=base)
    b[0, 3, 1], b[1, 3, 1], b[0, 7, rank - 1], b[1, 8, 0], b[1, 8, 1] = INF, -INF, -INF, INF, INF
    b[0, n - 1, 2] = float("nan")
    got = B.adapters(x, a, b, plan, scale=scale, base=base)
    w = want(x, a, b, base, index, scale)
    touched = torch.tensor([3, 7, 8, n - 1], device="cuda")
    keep = torch.ones(n, dtype=torch.bool, device="cuda")
    keep[touched] = False
    assert torch.equal(got[:, keep], clean[:, keep])
    special = ~w[:, touched].isfinite()
    assert bool((special.sum(0) > tokens // 6).all())
    assert torch.equal(got[:, touched].isnan(), w[:, touched].isnan())
    assert torch.equal(got[:, touched][special].nan_to_num(0.0, INF, -INF), w[:, touched][special].nan_to_num(0.0, INF, -INF))
    assert torch.equal(got[:, touched][~special], clean[:, touched][~special])


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("tokens,rank", [(3, 16), (20, 64), (40, 16), (300, 16), (300, 64), (300, 128)])
def test_inner_values_above_the_largest_bf16(tokens, rank, out):
    """3.4e38 is finite in 32 bits and rounds to infinity in bf16; infinite ones stay infinite."""
    import torch
    x, a = torch.ones(tokens, 8, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, rank, 8, dtype=torch.bfloat16, device="cuda")
    a[0, 1, 0], a[0, 2, 0] = 1, INF
    b = torch.zeros(1, 40, rank, dtype=torch.bfloat16, device="cuda")
    b[0, 1, 1], b[0, 2, 1], b[0, 3, 2], b[0, 4, 2] = 0.5, -2.0 ** -100, 3, -3
    b[0, 5:, 2] = 1
    plan = B.adapter_plan(torch.zeros(tokens, dtype=torch.int32, device="cuda"), 1)
    scale = torch.full((1,), 3.4e38, device="cuda")
    finite = a.clone()
    finite[0, 2, 0] = 0
    got = B.adapters(x, finite, b, plan, scale=scale, out_dtype=torch_types(out))
    v = float(scale[0])
    # v in 16 (24) bits, then the output's rounding
    tol = 2.0 ** -16 + 2.0 ** -8 if out == "bf16" else 2.0 ** -23
    assert bool((got[:, 0] == 0).all()) and bool((got[:, 3:] == 0).all())
    assert bool(((got[:, 1].double() / (v / 2) - 1).abs() <= tol).all()) and bool(((got[:, 2].double() / (-v * 2.0 ** -100) - 1).abs() <= tol).all())
    got = B.adapters(x, a, b, plan, scale=scale, out_dtype=torch_types(out))
    assert bool((got[:, 3] == INF).all()) and bool((got[:, 4] == -INF).all()) and bool((got[:, 5:] == INF).all())
    assert bool(got[:, :3].isnan().all())   # infinity times zero
