"""The linear layer's operators on the GPU against their 64-bit forms, at the
sizes, alignments and values where they can go wrong."""
from __future__ import annotations

import numpy as np
import pytest

import linear_ref as R
from shared_memory_tiled_gb300 import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from shared_memory_tiled_gb300 import build
    build.build()
    B.load()
    assert B.tr_device_status() == B.Status.OK
    yield
    assert B.tr_device_status() == B.Status.OK


def torch_types(name):
    import torch
    return {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn,
            "e5m2": torch.float8_e5m2}[name]


def on_gpu(x, kind, pitch=None, off=0):
    """x in `kind` on the GPU as a view of given row pitch that starts `off`
    elements into its buffer, the rest of which holds a sentinel; and the values
    it holds, in 64 bits."""
    import torch
    t = torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(torch_types(kind))
    rows, cols = x.shape
    pitch = pitch or cols
    buf = torch.full((off + rows * pitch + 16,), float("nan"), dtype=t.dtype, device="cuda")
    v = buf[off: off + rows * pitch].view(rows, pitch)[:, :cols] if rows else t.cuda()
    v.copy_(t)
    return v, t.to(torch.float64).numpy()


def host(t):
    import torch
    return t.to(torch.float64).cpu().numpy()


def codes(t):
    import torch
    return t.view(torch.uint8).cpu().numpy() if t.is_contiguous() else \
        torch.empty(t.shape, dtype=t.dtype, device=t.device).copy_(t).view(torch.uint8).cpu().numpy()


def close(got, want, bound, kind="f32"):
    tol = bound + (R.U16 * (np.abs(want) + bound) if kind == "bf16" else R.U32 * np.abs(want))
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (f"{bad.sum()} of {bad.size} outside, first at {np.argwhere(bad)[0]}: "
                           f"got {got[bad][0]!r} want {want[bad][0]!r} bound {tol[bad][0]!r}")


# --- quantize ----------------------------------------------------------------------

SHAPES = [(1, 1), (1, 128), (1, 4096), (2, 129), (127, 127), (128, 128), (129, 257), (300, 1000),
          (7, 8), (513, 15), (1000, 16)]


def values(rows, cols, seed):
    """Values of many magnitudes, with rows, columns and blocks of zeros, and
    values so small that the floor of the block maximum counts."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, cols)) * np.exp(3 * rng.standard_normal((rows, 1)))
    x[rng.random((rows, cols)) < 0.05] = 0
    if rows > 2:
        x[rows // 2] = 0
    if cols > 2:
        x[:, cols // 3] *= 1e-35
    if rows > 128 and cols > 128:
        x[:128, :128] = 0
    return x


def check_quant(x, kind, fp8, block, pitch=None, off=0):
    v, held = on_gpu(x, kind, pitch, off)
    q, s, qt, st = B.quantize_fp8(v, dtype=torch_types(fp8), block_rows=block, transposed=True)
    held = held.astype(np.float32)
    wq, ws = R.quantize(held, fp8, block)
    wt, wst = R.quantize(np.ascontiguousarray(held.T), fp8, block)

    def same(got, want):  # codes; a NaN has two, and the sign of a NaN says nothing
        nan = np.isnan(R.fp8_values(want, fp8))
        return np.array_equal(np.where(nan, 0, got), np.where(nan, 0, want)) and \
            np.isnan(R.fp8_values(got, fp8))[nan].all()

    assert np.array_equal(s.cpu().numpy(), ws, equal_nan=True)
    assert np.array_equal(st.cpu().numpy(), wst, equal_nan=True)
    assert same(codes(q), wq)
    assert same(codes(qt), wt)
    q1, s1 = B.quantize_fp8(v, dtype=torch_types(fp8), block_rows=block)
    assert np.array_equal(codes(q1), codes(q)) and np.array_equal(s1.cpu().numpy(), s.cpu().numpy(), equal_nan=True)


@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("fp8", ["e4m3", "e5m2"])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_quantize(kind, fp8, block):
    for i, (rows, cols) in enumerate(SHAPES):
        check_quant(values(rows, cols, i), kind, fp8, block)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_quantize_pitches_and_offsets(kind):
    x = values(200, 300, 5)
    for pitch, off in [(304, 0), (301, 0), (320, 1), (320, 3), (303, 2), (308, 4)]:
        check_quant(x, kind, "e4m3", 1, pitch, off)


@pytest.mark.parametrize("block", [1, 128])
def test_quantize_nan_and_infinity(block):
    x = values(260, 260, 9)
    x[3, 5], x[140, 200], x[200, 20] = np.nan, np.inf, -np.inf
    check_quant(x, "f32", "e4m3", block)
    check_quant(x, "f32", "e5m2", block)
    check_quant(x, "bf16", "e4m3", block)


def test_quantize_writes_nothing_between_rows():
    import torch
    rows, cols = 130, 70
    v, held = on_gpu(values(rows, cols, 3), "f32")
    q = torch.full((rows, 96), 0xAB, dtype=torch.uint8, device="cuda")
    qt = torch.full((cols, 144), 0xCD, dtype=torch.uint8, device="cuda")
    s = torch.full((1, rows + 5), -7.0, device="cuda")
    st = torch.full((2, cols + 3), -7.0, device="cuda")
    args = B.QuantizeArgs(v.data_ptr(), q.data_ptr(), s.data_ptr(), qt.data_ptr(), st.data_ptr(),
                          B.DType.F32, B.DType.E4M3, 1, 0, rows, cols, cols, 96, rows + 5, 144,
                          cols + 3, torch.cuda.current_stream().cuda_stream)
    B.check(B.tr_quantize_fp8(args))
    wq, ws = R.quantize(held.astype(np.float32), "e4m3", 1)
    assert np.array_equal(q[:, :cols].cpu().numpy(), wq) and bool((q[:, cols:] == 0xAB).all())
    assert bool((qt[:, rows:] == 0xCD).all())
    assert np.array_equal(s[:, :rows].cpu().numpy(), ws) and bool((s[:, rows:] == -7).all())
    assert bool((st[:, cols:] == -7).all())


# --- product -----------------------------------------------------------------------

def operand(rows, k, kind, block, seed):
    """8-bit operand (padded pitch, garbage between rows) and its codes and scales."""
    import torch
    rng = np.random.default_rng(seed)
    x = (rng.standard_normal((rows, k)) * np.exp(rng.standard_normal((rows, 1)))).astype(np.float32)
    q, s = R.quantize(x, kind, block)
    pitch = -(-k // 16) * 16 + 16 * (seed % 2)
    buf = torch.full((rows, pitch), 0x7E, dtype=torch.uint8, device="cuda")
    buf[:, :k] = torch.from_numpy(q)
    return buf.view(torch_types(kind))[:, :k], torch.from_numpy(s).cuda(), q, s


def check_product(m, n, k, ka="e4m3", kb="e4m3", ab=1, bb=128, kind="bf16", seed=0, out=None,
                  accumulate=False):
    import torch
    a, sa, qa, ha = operand(m, k, ka, ab, seed)
    b, sb, qb, hb = operand(n, k, kb, bb, seed + 1)
    want, bound = R.matmul(qa, ha, ka, ab, qb, hb, kb, bb)
    if accumulate:
        old = host(out)
        want, bound = want + old, bound + R.U32 * (np.abs(old) + np.abs(want))
    got = B.matmul_fp8(a, sa, b, sb, out=out, out_dtype=None if out is not None else torch_types(kind),
                       accumulate=accumulate)
    close(host(got), want, bound, kind)
    return got


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("m,n,k", [
    (1, 1, 1), (1, 128, 128), (1, 1000, 4096), (16, 129, 200), (17, 64, 1111), (33, 300, 2048),
    (64, 512, 640), (65, 128, 128), (128, 128, 256), (129, 127, 127), (300, 700, 1000),
    (257, 2049, 1111), (1000, 130, 8192)])
def test_product(m, n, k, kind):
    check_product(m, n, k, kind=kind, seed=m + n + k)


@pytest.mark.parametrize("m", [1, 40, 200])
@pytest.mark.parametrize("ab,bb", [(1, 1), (1, 128), (128, 1), (128, 128)])
@pytest.mark.parametrize("ka,kb", [("e4m3", "e5m2"), ("e5m2", "e4m3"), ("e5m2", "e5m2")])
def test_product_types_and_blocks(m, ab, bb, ka, kb):
    check_product(m, 333, 1500, ka, kb, ab, bb, "f32", seed=m)


@pytest.mark.parametrize("ab,bb", [(1, 1), (1, 128), (128, 1), (128, 128)])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_large_product(ab, bb, kind):
    """Tiles of 256 x 256, whole and at the edges, contractions of one block and of
    more than the ring holds, more tiles than pairs of CTAs."""
    check_product(2304, 2304, 128, "e4m3", "e4m3", ab, bb, kind, seed=1)
    check_product(2304, 2304, 1536, "e5m2", "e4m3", ab, bb, kind, seed=2)
    check_product(2435, 2311, 777, "e4m3", "e4m3", ab, bb, kind, seed=3)
    check_product(130, 20000, 300, "e4m3", "e4m3", ab, bb, kind, seed=4)


def test_large_product_into_a_view_and_accumulated():
    import torch
    m, n, k = 2310, 2300, 520
    for kind in ("bf16", "f32"):
        for pitch, off in [(n, 0), (n + 3, 1), (n + 4, 8)]:
            buf = torch.full((off + m * pitch + 8,), -3.0, dtype=torch_types(kind), device="cuda")
            view = buf[off: off + m * pitch].view(m, pitch)[:, :n]
            check_product(m, n, k, kind=kind, seed=m, out=view)
            check_product(m, n, k, kind=kind, seed=m + 2, out=view, accumulate=True)
            view.fill_(-3.0)
            assert bool((buf == -3.0).all())


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("m", [3, 150])
def test_product_into_a_view_and_accumulated(m, kind):
    import torch
    n, k = 200, 900
    for pitch, off in [(200, 0), (203, 1), (208, 8)]:
        buf = torch.full((off + m * pitch + 8,), -3.0, dtype=torch_types(kind), device="cuda")
        view = buf[off: off + m * pitch].view(m, pitch)[:, :n]
        check_product(m, n, k, kind=kind, seed=m, out=view)
        check_product(m, n, k, kind=kind, seed=m + 2, out=view, accumulate=True)
        rest = buf.clone()
        rest[off: off + m * pitch].view(m, pitch)[:, :n] = -3.0
        assert bool((rest == -3.0).all())


def test_product_without_a_contraction():
    import torch
    a = torch.empty(5, 0, dtype=torch.float8_e4m3fn, device="cuda")
    b = torch.empty(7, 0, dtype=torch.float8_e4m3fn, device="cuda")
    sa, sb = torch.empty(0, 5, device="cuda"), torch.empty(0, 7, device="cuda")
    out = torch.full((5, 7), 2.0, device="cuda")
    B.matmul_fp8(a, sa, b, sb, out=out, accumulate=True)
    assert bool((out == 2).all())
    assert bool((B.matmul_fp8(a, sa, b, sb, out=out) == 0).all())


def test_product_nan_scale_reaches_its_rows_only():
    import torch
    m, n, k = 150, 140, 300
    a, sa, *_ = operand(m, k, "e4m3", 1, 1)
    b, sb, *_ = operand(n, k, "e4m3", 128, 2)
    sa[1, 77] = float("nan")
    got = B.matmul_fp8(a, sa, b, sb, out_dtype=torch.float32)
    assert bool(got[77].isnan().all())
    assert not bool(got[:77].isnan().any()) and not bool(got[78:].isnan().any())


def test_product_repeats_bit_for_bit():
    a, sa, *_ = operand(7, 4096, "e4m3", 1, 1)
    b, sb, *_ = operand(512, 4096, "e4m3", 128, 2)
    first = B.matmul_fp8(a, sa, b, sb)
    for _ in range(20):
        assert bool((B.matmul_fp8(a, sa, b, sb) == first).all())


# --- layer norm --------------------------------------------------------------------

LN = [(1, 1), (1, 7), (3, 128), (5, 1000), (2, 1024), (9, 2047), (4, 4099), (3, 8192), (2, 16384),
      (2, 20001), (1, 33000), (1, 70001), (300, 96)]


def rows_of(rows, cols, seed, offset=3.0):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, cols)) * np.exp(rng.standard_normal((rows, 1))) + offset
    if rows > 2:
        x[1] = 2.5          # no variance
    return x


@pytest.mark.parametrize("wkind", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_layernorm(kind, wkind):
    for i, (rows, cols) in enumerate(LN):
        check_layernorm(rows, cols, kind, wkind, i)
        check_layernorm(rows, cols, kind, wkind, i, bias=False)


def check_layernorm(rows, cols, kind, wkind, seed, bias=True, pitch=None, off=0, out=None):
    x, held = on_gpu(rows_of(rows, cols, seed), kind, pitch, off)
    rng = np.random.default_rng(seed + 100)
    gamma, hg = on_gpu(1 + 0.1 * rng.standard_normal((1, cols)), wkind)
    beta, hb = on_gpu(rng.standard_normal((1, cols)), wkind)
    y, mean, rstd = B.layernorm(x, gamma[0], beta[0] if bias else None, out=out)
    wy, wm, wr, by, bm, br = R.layernorm(held, hg, hb if bias else None, 1e-5)
    close(host(mean), wm, bm)
    close(host(rstd), wr, br)
    close(host(y), wy, by, kind)


def check_layernorm_backward(rows, cols, kind, wkind, seed, bias=True, pitch=None, off=0, out=None):
    import torch
    x, held = on_gpu(rows_of(rows, cols, seed), kind, pitch, off)
    rng = np.random.default_rng(seed + 100)
    dy, hd = on_gpu(rng.standard_normal((rows, cols)), kind, pitch, off)
    gamma, hg = on_gpu(1 + 0.1 * rng.standard_normal((1, cols)), wkind)
    _, mean, rstd, *_ = R.layernorm(held, hg, None, 1e-5)
    tm, tr = (torch.from_numpy(v.astype(np.float32)).cuda() for v in (mean, rstd))
    dx, dg, db = B.layernorm_backward(dy, x, gamma[0], tm, tr, bias=bias, out=out)
    wx, wg, wb, bx, bg, bb = R.layernorm_backward(hd, held, hg, tm.cpu().numpy(), tr.cpu().numpy())
    close(host(dx), wx, bx, kind)
    close(host(dg), wg, bg)
    if bias:
        close(host(db), wb, bb)
    else:
        assert db is None


@pytest.mark.parametrize("wkind", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_layernorm_backward(kind, wkind):
    for i, (rows, cols) in enumerate(LN + [(1500, 200), (700, 1025)]):
        check_layernorm_backward(rows, cols, kind, wkind, i)
    check_layernorm_backward(40, 500, kind, wkind, 77, bias=False)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_layernorm_pitches_and_offsets(kind):
    import torch
    for rows, cols in [(40, 300), (5, 5000)]:
        for pitch, off in [(cols + 4, 0), (cols + 1, 0), (cols + 16, 1), (cols + 16, 3), (cols + 3, 2)]:
            check_layernorm(rows, cols, kind, "f32", 1, pitch=pitch, off=off)
            check_layernorm_backward(rows, cols, kind, "f32", 1, pitch=pitch, off=off)
            # an output that is offset otherwise than its input, and nothing written beside it
            buf = torch.full((7 + rows * (cols + 5),), -3.0, dtype=torch_types(kind), device="cuda")
            view = buf[7:].view(rows, cols + 5)[:, :cols]
            check_layernorm(rows, cols, kind, "f32", 2, pitch=pitch, off=off, out=view)
            check_layernorm_backward(rows, cols, kind, "f32", 2, pitch=pitch, off=off, out=view)
            view.fill_(-3.0)
            assert bool((buf == -3.0).all())


def test_layernorm_large_offset_keeps_its_variance():
    check_layernorm(6, 4096, "f32", "f32", 3)
    x, held = on_gpu(rows_of(4, 2048, 4, offset=10000.0), "f32")
    gamma, hg = on_gpu(np.ones((1, 2048)), "f32")
    y, mean, rstd = B.layernorm(x, gamma[0])
    wy, wm, wr, by, bm, br = R.layernorm(held, hg, None, 1e-5)
    close(host(rstd), wr, br)
    close(host(y), wy, by)


def test_layernorm_nan_and_infinity_stay_in_their_rows():
    import torch
    x = torch.randn(8, 1000, device="cuda")
    x[2, 3], x[5, 999] = float("nan"), float("inf")
    y, mean, rstd = B.layernorm(x, torch.ones(1000, device="cuda"))
    bad = y.isnan().all(1)
    assert bad.tolist() == [False, False, True, False, False, True, False, False]
    assert not bool(y[~bad].isnan().any())


def test_layernorm_backward_without_rows():
    import torch
    x = torch.empty(0, 50, device="cuda")
    v = torch.empty(0, device="cuda")
    dx, dg, db = B.layernorm_backward(x, x, torch.ones(50, device="cuda"), v, v)
    assert dx.shape == (0, 50) and bool((dg == 0).all()) and bool((db == 0).all())


def test_layernorm_backward_repeats_bit_for_bit():
    import torch
    x, dy = torch.randn(3000, 513, device="cuda"), torch.randn(3000, 513, device="cuda")
    gamma = torch.randn(513, device="cuda")
    _, mean, rstd = B.layernorm(x, gamma)
    first = B.layernorm_backward(dy, x, gamma, mean, rstd)
    for _ in range(10):
        for a, b in zip(B.layernorm_backward(dy, x, gamma, mean, rstd), first):
            assert torch.equal(a, b)


# --- streams, graphs ---------------------------------------------------------------

def chain(x, gamma, beta, w, stream=None):
    """Forward: norm, quantize, product; backward of a sum: the other two products."""
    y, mean, rstd = B.layernorm(x, gamma, beta, stream=stream)
    q, s, qt, st = B.quantize_fp8(y, transposed=True, stream=stream)
    wq, ws, wt, wst = B.quantize_fp8(w, block_rows=128, transposed=True, stream=stream)
    out = B.matmul_fp8(q, s, wq, ws, stream=stream)
    dq, ds, dt, dst = B.quantize_fp8(out, transposed=True, stream=stream)
    dw = B.matmul_fp8(dt, dst, qt, st, out_dtype=w.dtype, stream=stream)
    dy = B.matmul_fp8(dq, ds, wt, wst, stream=stream)
    return (out, dw) + B.layernorm_backward(dy, x, gamma, mean, rstd, stream=stream)


def inputs():
    import torch
    torch.manual_seed(0)
    return (torch.randn(300, 512, device="cuda", dtype=torch.bfloat16), torch.randn(512, device="cuda"),
            torch.randn(512, device="cuda"), torch.randn(200, 512, device="cuda"))


def test_another_stream_gives_the_same():
    import torch
    args = inputs()
    want = chain(*args)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        got = chain(*args, stream=s.cuda_stream)
        s.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_chain_replays_from_a_graph():
    import torch
    args = inputs()
    want = chain(*args)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        chain(*args)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        got = chain(*args)
    for _ in range(3):
        for t in got:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
