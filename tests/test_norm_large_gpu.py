"""Root-mean-square norm, its backward pass and the adapters where offsets in elements pass 32 bits."""
from __future__ import annotations

import pytest

from shared_memory_tiled_gb300 import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from shared_memory_tiled_gb300 import build
    build.build()
    B.load()
    yield
    assert B.tr_device_status() == B.Status.OK


@pytest.mark.parametrize("rows,cols", [(270000, 8192), (2200000, 1001), (75003, 30000), (110000, 20001)])
def test_last_rows(rows, cols):
    """Of more than 2^31 values the last rows (from a multiple of 128 on) are bit for bit those of a call on them alone: both
    take the same kernel, and a row's sums depend on its length only."""
    import torch
    assert rows * cols > 2 ** 31
    x, res = (torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda").normal_() for _ in range(2))
    gamma = torch.rand(cols, device="cuda") + 0.5
    at = slice((rows - 500) // 128 * 128, rows)
    q, s, qt, st, h, rstd = B.rmsnorm_fp8(x, gamma, res, transposed=True)
    alone = B.rmsnorm_fp8(x[at], gamma, res[at], transposed=True)
    for a, b in zip((q[at], s[:, at], qt[:, at], st[at.start // 128:], h[at], rstd[at]), alone):
        assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))
    del q, s, qt, st, x
    dy = torch.empty_like(res).normal_()
    dx, dgamma = B.rmsnorm_backward(dy, h, gamma, rstd, dresidual=res)
    dx1, _ = B.rmsnorm_backward(dy[at], h[at], gamma, rstd[at], dresidual=res[at])
    want, size = (torch.zeros(cols, dtype=torch.float64, device="cuda") for _ in range(2))
    for i in range(0, rows, 20000):
        part = dy[i:i + 20000].double() * h[i:i + 20000] * rstd[i:i + 20000, None]
        want += part.sum(0)
        size += part.abs().sum(0)
    assert torch.equal(dx[at], dx1)
    assert bool(((dgamma - want).abs() <= (rows + 8) * 2 ** -24 * size).all())


# few tokens, both kernels, many tokens; outputs on and off 16-byte boundaries
@pytest.mark.parametrize("n", [264, 265])
@pytest.mark.parametrize("tokens,pitch", [(40, 1 << 26), (700, 1 << 22), (3000, 1 << 20)])
def test_adapters_far_rows(tokens, pitch, n):
    import torch
    assert tokens * pitch > 2 ** 31
    wide, far = (torch.empty(tokens, pitch, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    x, base, out = wide[:, 8:144].normal_(), wide[:, 1024:1024 + n].normal_(), far[:, pitch - 320:pitch - 320 + n]
    a, b = torch.randn(3, 16, 136, device="cuda").bfloat16(), torch.randn(3, n, 16, device="cuda").bfloat16()
    plan = B.adapter_plan((torch.arange(tokens, device="cuda") % 4 - 1).int(), 3)
    B.adapters(x, a, b, plan, base=base, out=out)
    assert torch.equal(out, B.adapters(x.contiguous(), a, b, plan, base=base.contiguous()))


@pytest.mark.parametrize("tokens", [20, 500, 3000])
def test_adapters_far_planes(tokens):
    import torch
    g = torch.Generator(device="cuda").manual_seed(tokens)
    a = torch.empty(600, 128, 32768, dtype=torch.bfloat16, device="cuda")[:, :, :136].random_(-2, 3, generator=g)
    b = torch.empty(600, 264, 16384, dtype=torch.bfloat16, device="cuda")[:, :, :128].random_(-2, 3, generator=g)
    assert a.stride(0) * 599 > 2 ** 31 and b.stride(0) * 599 > 2 ** 31
    x = torch.randint(-2, 3, (tokens, 136), device="cuda", generator=g).bfloat16()   # whole numbers: exact in any order
    index = torch.arange(tokens, device="cuda", dtype=torch.int32) % 3 + 597
    got = B.adapters(x, a, b, B.adapter_plan(index, 600))
    for i in range(597, 600):
        at = index == i
        want = x[at].double() @ a[i].double().t() @ b[i].double().t()
        assert torch.equal(got[at], want.bfloat16())
