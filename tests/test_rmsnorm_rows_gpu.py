"""Root-mean-square norm where a block (or a warp) holds rows in registers and takes a second one: against the 64-bit form,
and bit for bit against the same rows in calls that give each block one."""
from __future__ import annotations

import numpy as np
import pytest

import norm_ref as N
from shared_memory_tiled_gb300 import binding as B
from test_linear_gpu import close, codes, host, torch_types

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from shared_memory_tiled_gb300 import build
    build.build()
    B.load()
    yield
    assert B.tr_device_status() == B.Status.OK


# more rows than SMs and at most twice as many, up to 2048 chunks of 16 bytes; a warp's rows in more blocks than are resident
SHAPES = [(256, 8192, "bf16"), (200, 3000, "bf16"), (290, 16384, "bf16"), (300, 2048, "bf16"), (230, 4096, "f32"), (280, 8192, "f32"), (300, 516, "f32"),
          (6000, 1024, "bf16"), (6000, 512, "f32"), (40000, 128, "bf16"), (40000, 104, "f32")]


@pytest.mark.parametrize("add", [True, False])
@pytest.mark.parametrize("rows,cols,kind", SHAPES)
def test_second_rows(rows, cols, kind, add):
    import torch
    g = torch.Generator(device="cuda").manual_seed(rows + cols)
    x, res = (torch.randn(rows, cols, device="cuda", generator=g).to(torch_types(kind)) for _ in range(2))
    res = res if add else None
    gamma = torch.rand(cols, device="cuda", generator=g) + 0.5
    y = torch.empty_like(x)
    q, s, h, rstd = B.rmsnorm_fp8(x, gamma, res, out=y)
    want_h = x if res is None else (x.float() + res.float()).to(x.dtype)
    assert torch.equal(h, want_h)
    wy, wr, ey, er = N.rmsnorm(host(want_h), host(gamma), 1e-6)
    close(host(rstd), wr, er)
    close(host(y), wy, ey, kind)
    N.check_quantized(codes(q), s.cpu().numpy(), wy, ey, "e4m3")
    y1, h1, rstd1 = B.rmsnorm(x, gamma, res)
    assert torch.equal(y1, y) and torch.equal(h1, h) and torch.equal(rstd1, rstd)
    for lo in list(range(0, rows, 100))[-7:]:
        at = slice(lo, lo + 100)
        p, t, _, r = B.rmsnorm_fp8(x[at], gamma, None if res is None else res[at])
        assert torch.equal(r, rstd[at]) and np.array_equal(codes(p), codes(q[at])) and torch.equal(t, s[:, at])
