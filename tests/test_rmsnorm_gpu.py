"""Root-mean-square norm, its 8-bit output and its backward pass on the GPU against their 64-bit
forms, at the sizes, alignments and values where they can go wrong."""
from __future__ import annotations

import numpy as np
import pytest

import norm_ref as N
from shared_memory_tiled_gb300 import binding as B
from test_linear_gpu import close, codes, host, on_gpu, torch_types

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from shared_memory_tiled_gb300 import build
    build.build()
    B.load()
    assert B.tr_device_status() == B.Status.OK
    yield
    assert B.tr_device_status() == B.Status.OK


# rows, cols, pitch, elements before the first value: both sides of the limits between the kernels
# (chunks to a thread, threads to a row, what a ring of rows holds), and rows off 16-byte boundaries
SHAPES = [(1, 1, None, 0), (1, 8192, None, 0), (2, 7, 9, 1), (3, 128, None, 0), (5, 129, 136, 0), (130, 1000, 1000, 0), (300, 1024, 1024, 0),
          (129, 1025, 1027, 3), (700, 2048, 2056, 8), (600, 513, 513, 0), (37, 8184, 8184, 0), (21, 8200, 8200, 0), (9, 16384, 16384, 0),
          (7, 16392, 16392, 0), (5, 11569, 11569, 0), (3, 20001, 20003, 5), (4, 40000, 40000, 0), (260, 96, 101, 2)]


def inputs(rows, cols, seed):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, cols)) * np.exp(rng.standard_normal((rows, 1)))
    res = rng.standard_normal((rows, cols)) * 3
    if rows > 2:
        x[1], res[1] = 0, 0                 # a row of zeros: rstd is 1 / sqrt(eps)
    if cols > 300:
        x[-1, 128:256], res[-1, 128:256] = 0, 0   # a block of zeros
    return x, res, 1 + 0.2 * rng.standard_normal(cols)


def stream(x, res, kind):
    import torch
    h = x if res is None else (x.float() + res.float()).to(torch_types(kind))
    return h, h.to(torch.float64).cpu().numpy()


@pytest.mark.parametrize("wkind", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("add", [True, False])
def test_forward(kind, wkind, add):
    import torch
    for i, (rows, cols, pitch, off) in enumerate(SHAPES):
        x, res, gamma = inputs(rows, cols, i)
        x, _ = on_gpu(x, kind, pitch, off)
        res = on_gpu(res, kind, pitch, off + (i % 3 if off else 0))[0] if add else None
        gamma, wide = on_gpu(gamma[None], wkind, off=off % 2)
        y, h, rstd = B.rmsnorm(x, gamma[0], res, eps=1e-5)
        want_h, wide_h = stream(x, res, kind)
        assert torch.equal(h, want_h) and (add or h is x)
        wy, wr, ey, er = N.rmsnorm(wide_h, wide[0], 1e-5)
        close(host(y), wy, ey, kind)
        close(host(rstd), wr, er)


@pytest.mark.parametrize("fp8", ["e4m3", "e5m2"])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_8_bits(kind, fp8):
    import torch
    for i, (rows, cols, pitch, off) in enumerate(SHAPES):
        x, res, gamma = inputs(rows, cols, 50 + i)
        x, _ = on_gpu(x, kind, pitch, off)
        res = on_gpu(res, kind, pitch, off)[0] if i % 2 else None
        gamma, wide = on_gpu(gamma[None], "f32")
        want_h, wide_h = stream(x, res, kind)
        wy, wr, ey, er = N.rmsnorm(wide_h, wide[0], 1e-6)
        y = torch.empty(rows, cols, dtype=x.dtype, device="cuda")
        q, s, qt, st, h, rstd = B.rmsnorm_fp8(x, gamma[0], res, dtype=torch_types(fp8), transposed=True, out=y)
        assert torch.equal(h, want_h)
        close(host(rstd), wr, er)
        close(host(y), wy, ey, kind)
        N.check_quantized(codes(q), s.cpu().numpy(), wy, ey, fp8)
        N.check_quantized(codes(qt), st.cpu().numpy(), wy.T, ey.T, fp8)
        q1, s1, h1, rstd1 = B.rmsnorm_fp8(x, gamma[0], res, dtype=torch_types(fp8))
        assert np.array_equal(codes(q1), codes(q)) and torch.equal(s1, s) and torch.equal(h1, h) and torch.equal(rstd1, rstd)
        y1, _, _ = B.rmsnorm(x, gamma[0], res)
        assert torch.equal(y1, y)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_stream_in_place_and_what_lies_beside(kind):
    """The new stream in the residual's place; nothing outside the outputs is written."""
    import torch
    for rows, cols, pitch, off in [(70, 1000, 1003, 1), (40, 512, 520, 8), (3, 20001, 20003, 5)]:
        x, res, gamma = inputs(rows, cols, rows)
        x, _ = on_gpu(x, kind)
        res, _ = on_gpu(res, kind, pitch, off)
        gamma = torch.from_numpy(gamma).float().cuda()
        want = B.rmsnorm(x, gamma, res)
        buf = torch.full((off + rows * pitch + 16,), 7.0, dtype=x.dtype, device="cuda")
        in_place = buf[off:off + rows * pitch].view(rows, pitch)[:, :cols]
        in_place.copy_(res)
        out = torch.full((off + rows * pitch + 16,), 7.0, dtype=x.dtype, device="cuda")
        y, h, rstd = B.rmsnorm(x, gamma, in_place, out=out[off:off + rows * pitch].view(rows, pitch)[:, :cols], residual_out=in_place)
        assert h is in_place
        for got, w in zip((y, h, rstd), want):
            assert torch.equal(got, w)
        for b in (buf, out):
            assert bool((b[:off] == 7).all()) and bool((b[off + rows * pitch:] == 7).all())
            assert bool((b[off:off + rows * pitch].view(rows, pitch)[:, cols:] == 7).all())


def test_large_values_nan_and_infinity():
    import torch
    x = torch.randn(6, 300, device="cuda").bfloat16()
    x[0, 3], x[1, 5], x[2, 200] = float("nan"), float("inf"), float("-inf")
    x[3] = 1e18   # squares of 1e36 and their sum stay in range
    gamma = torch.ones(300, device="cuda")
    q, s, qt, st, _, rstd = B.rmsnorm_fp8(x, gamma, transposed=True)
    y, _, _ = B.rmsnorm(x, gamma)
    assert bool(y[0].isnan().all()) and bool(rstd[0].isnan())
    assert bool((rstd[1:3] == 0).all())              # 1 / infinity; infinity * 0 is NaN
    assert bool(y[1, 5].isnan()) and bool((y[1, :5] == 0).all()) and bool(y[2, 200].isnan())
    assert bool(((y[3].float() - 1).abs() <= 2 ** -8).all())
    assert bool(s[:, 0].isnan().all()) and bool(s[0, 1].isnan()) and bool(s[1, 2].isnan())
    assert bool(q[0].float().isnan().all()) and bool(q[1, :128].float().isnan().all())
    assert bool((q[1, 128:].float() == 0).all()) and bool((q[4:].float().abs() <= 448).all())
    assert bool(st.isnan().all()) and bool(qt[0].float().isnan().all())   # the row of NaN is in every column's block


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("add", [True, False])
def test_backward(kind, add):
    import torch
    for i, (rows, cols, pitch, off) in enumerate(SHAPES):
        h, dres, gamma = inputs(rows, cols, 90 + i)
        dy = np.random.default_rng(i).standard_normal((rows, cols)) * 1e-2
        h, wh = on_gpu(h, kind, pitch, off)
        dy, wdy = on_gpu(dy, kind, pitch, off + (i % 2 if off else 0))
        dres, wres = on_gpu(dres * 1e-2, kind, pitch, off) if add else (None, None)
        gamma, wg = on_gpu(gamma[None], ["f32", "bf16"][i % 2])
        rstd = torch.from_numpy(N.rmsnorm(wh, wg[0], 1e-4)[1]).float().cuda()
        dx, dgamma = B.rmsnorm_backward(dy, h, gamma[0], rstd, dresidual=dres)
        wx, ww, ex, ew = N.rmsnorm_backward(wdy, wh, wg[0], host(rstd), wres)
        close(host(dx), wx, ex, kind)
        close(host(dgamma), ww, ew)
        again = B.rmsnorm_backward(dy, h, gamma[0], rstd, dresidual=dres)
        assert torch.equal(again[0], dx) and torch.equal(again[1], dgamma)
        if add:  # in dresidual's place
            dx2, _ = B.rmsnorm_backward(dy, h, gamma[0], rstd, dresidual=dres, out=dres)
            assert torch.equal(dx2, dx)


def test_backward_many_rows():
    """More rows than resident blocks hold at one time, of each length."""
    import torch
    for rows, cols in [(5000, 256), (3001, 1000), (1300, 8192), (700, 9000)]:
        g = torch.Generator(device="cuda").manual_seed(rows)
        h, dy, dres = (torch.randn(rows, cols, device="cuda", generator=g).bfloat16() for _ in range(3))
        gamma = torch.rand(cols, device="cuda", generator=g) + 0.5
        y, _, rstd = B.rmsnorm(h, gamma)
        wy, wr, ey, er = N.rmsnorm(host(h), host(gamma), 1e-6)
        close(host(y), wy, ey, "bf16")
        close(host(rstd), wr, er)
        dx, dgamma = B.rmsnorm_backward(dy, h, gamma, rstd, dresidual=dres)
        wx, ww, ex, ew = N.rmsnorm_backward(host(dy), host(h), host(gamma), host(rstd), host(dres))
        close(host(dx), wx, ex, "bf16")
        close(host(dgamma), ww, ew)


def test_8_bits_many_rows():
    import torch
    for rows, cols, kind in [(5000, 256, "bf16"), (3001, 1000, "f32"), (1300, 8192, "bf16"), (2000, 519, "f32"), (1025, 8200, "bf16"),
                             (1100, 5000, "f32"), (1023, 4096, "bf16")]:
        g = torch.Generator(device="cuda").manual_seed(rows)
        x, res = (torch.randn(rows, cols, device="cuda", generator=g).to(torch_types(kind)) for _ in range(2))
        gamma = torch.rand(cols, device="cuda", generator=g) + 0.5
        q, s, qt, st, h, rstd = B.rmsnorm_fp8(x, gamma, res, transposed=True)
        want_h, wide_h = stream(x, res, kind)
        assert torch.equal(h, want_h)
        wy, wr, ey, er = N.rmsnorm(wide_h, host(gamma), 1e-6)
        close(host(rstd), wr, er)
        N.check_quantized(codes(q), s.cpu().numpy(), wy, ey, "e4m3")
        N.check_quantized(codes(qt), st.cpu().numpy(), wy.T, ey.T, "e4m3")


def test_no_rows_and_no_columns():
    import torch
    gamma = torch.ones(9, device="cuda")
    none = torch.empty(0, 9, device="cuda")
    y, h, rstd = B.rmsnorm(none, gamma, none)
    assert y.shape == h.shape == (0, 9) and rstd.shape == (0,)
    dx, dgamma = B.rmsnorm_backward(none, none, gamma, rstd)
    assert dx.shape == (0, 9) and bool((dgamma == 0).all())
    y, h, rstd = B.rmsnorm(torch.empty(70, 0, device="cuda"), gamma[:0])
    assert y.shape == (70, 0) and bool(rstd.isnan().all())
    q, s, qt, st, h, rstd = B.rmsnorm_fp8(torch.empty(70, 0, device="cuda"), gamma[:0], transposed=True)
    assert q.shape == (70, 0) and qt.shape == (0, 70) and s.numel() == st.numel() == 0 and bool(rstd.isnan().all())


def test_other_stream_and_graph():
    """A captured and replayed step on a side stream gives the eager call's bits on new inputs."""
    import torch
    x, res, dy = (torch.randn(300, 1000, device="cuda").bfloat16() for _ in range(3))
    gamma = torch.rand(1000, device="cuda")

    def step(stream=None):
        q, s, qt, st, h, rstd = B.rmsnorm_fp8(x, gamma, res, transposed=True, stream=stream)
        return [q, s, qt, st, h, rstd, *B.rmsnorm_backward(dy, h, gamma, rstd, dresidual=res, stream=stream)]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    x.normal_()
    res.normal_()
    graph.replay()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    eager = step(side.cuda_stream)
    torch.cuda.synchronize()
    for a, b in zip(held, eager):
        assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def test_refusals():
    import torch
    x, gamma = torch.randn(4, 6, device="cuda"), torch.ones(6, device="cuda")
    with pytest.raises(ValueError):
        B.rmsnorm(x.cpu(), gamma)
    with pytest.raises(ValueError):
        B.rmsnorm(x, gamma[:5])
    with pytest.raises(ValueError):
        B.rmsnorm(x, gamma, x[:3])
    with pytest.raises(ValueError):
        B.rmsnorm(x, gamma, x.bfloat16())
    with pytest.raises(ValueError):
        B.rmsnorm(x, gamma, residual_out=torch.empty_like(x))
    with pytest.raises(ValueError):
        B.rmsnorm(x.t(), torch.ones(4, device="cuda"))
    with pytest.raises(TypeError):
        B.rmsnorm(x.half(), gamma)
    with pytest.raises(TypeError):
        B.rmsnorm_fp8(x, gamma, dtype=torch.float32)
    with pytest.raises(B.TransposeError):
        B.rmsnorm(x, gamma, out=x)
    with pytest.raises(B.TransposeError):
        B.rmsnorm(x, gamma, eps=-1.0)
    rstd = torch.ones(4, device="cuda")
    with pytest.raises(ValueError):
        B.rmsnorm_backward(x, x, gamma, rstd[:3])
    with pytest.raises(ValueError):
        B.rmsnorm_backward(x.bfloat16(), x, gamma, rstd)
    with pytest.raises(ValueError):
        B.rmsnorm_backward(x, x, gamma, rstd, dresidual=x[:2])
    with pytest.raises(B.TransposeError):
        B.rmsnorm_backward(x, x, gamma, rstd, out=x)
