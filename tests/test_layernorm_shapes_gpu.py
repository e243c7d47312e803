"""Layer norm at the sizes where batches run it: every shape of the kernel that keeps
the weights in shared memory, and backward passes whose blocks go round their ring
of rows more than twice.  The 64-bit forms run on the GPU here: they are the same
formulas and bounds as ``linear_ref``'s, on matrices of up to 80 million values."""
from __future__ import annotations

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


def sms():
    import torch
    return torch.cuda.get_device_properties(0).multi_processor_count


def types(name):
    import torch
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def matrix(rows, cols, kind, pitch, off, gen, offset=0.0, scale=True):
    """A view of the given pitch that starts `off` elements into a buffer of NaNs."""
    import torch
    buf = torch.full((off + rows * pitch,), float("nan"), dtype=types(kind), device="cuda")
    view = buf[off:].view(rows, pitch)[:, :cols]
    x = torch.randn(rows, cols, device="cuda", generator=gen)
    if scale:
        x.mul_(torch.exp(torch.randn(rows, 1, device="cuda", generator=gen)))
    view.copy_(x.add_(offset))
    return view


def target(rows, cols, kind, pitch, off):
    """An output laid out alike, in a buffer of sentinels; and the buffer."""
    import torch
    buf = torch.full((off + rows * pitch,), -3.0, dtype=types(kind), device="cuda")
    return buf[off:].view(rows, pitch)[:, :cols], buf


def close(got, want, bound, kind="f32"):
    tol = bound + (R.U16 * (want.abs() + bound) if kind == "bf16" else R.U32 * want.abs())
    bad = ~((got.double() - want).abs() <= tol)
    if bool(bad.any()):
        at = bad.nonzero()[0].tolist()
        raise AssertionError(f"{int(bad.sum())} of {bad.numel()} outside, first at {at}: got {got[tuple(at)].item()!r} "
                             f"want {want[tuple(at)].item()!r} bound {tol[tuple(at)].item()!r}")


# --- forward: 32 rows to an SM and more ------------------------------------------------

def forward_case(kind, wkind, rows, cols, pitch, off, bias):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(rows + 3 * cols + off)
    x = matrix(rows, cols, kind, pitch, off, gen, offset=3.0)
    x[1] = 2.5  # no variance
    gamma = (1 + 0.1 * torch.randn(cols, device="cuda", generator=gen)).to(types(wkind))
    beta = torch.randn(cols, device="cuda", generator=gen).to(types(wkind)) if bias else None
    out, buf = target(rows, cols, kind, pitch, off)
    y, mean, rstd = B.layernorm(x, gamma, beta, out=out)
    v, g = x.double(), gamma.double()
    wm = v.mean(1, keepdim=True)
    dev = v - wm
    wr = ((dev * dev).mean(1, keepdim=True) + 1e-5) ** -0.5
    wy = dev * wr * g + (0 if beta is None else beta.double())
    # as linear_ref.layernorm: a thread's own values, then ten levels of a tree
    depth = 64 + cols / 256
    dm = depth * R.U32 * v.abs().mean(1, keepdim=True) + R.U32 * wm.abs()
    dev = dev.abs_()
    dv = (depth + 4) * R.U32 * (dev ** 2).mean(1, keepdim=True) + 2 * dev.mean(1, keepdim=True) * dm + dm ** 2
    dr = wr * (0.5 * dv * wr ** 2 + 4 * R.U32)
    dy = g.abs() * (wr * (dm + R.U32 * dev) + dev * dr + 4 * R.U32 * dev * wr) + 2 * R.U32 * wy.abs()
    close(mean, wm[:, 0], dm[:, 0])
    close(rstd, wr[:, 0], dr[:, 0])
    close(y, wy, dy, kind)
    out.fill_(-3.0)
    assert bool((buf == -3.0).all())


@pytest.mark.parametrize("chunks", [128, 256, 512, 1024, 2048])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_forward_on_both_sides_of_each_shapes_limit(kind, chunks):
    """`chunks` 16-byte chunks are the most that one shape takes; the rows fill every
    group of every block and leave some groups a row short."""
    v = 8 if kind == "bf16" else 4
    rows = 32 * sms() + 37
    for cols in (chunks * v - v, chunks * v, chunks * v + v):
        forward_case(kind, "f32", rows, cols, cols, 0, True)
        forward_case(kind, "bf16", rows, cols, cols + v, 0, False)
        forward_case(kind, "bf16", rows, cols, cols + 1, 3, True)      # another shift in each row
    forward_case(kind, "f32", rows, chunks * v - 3, chunks * v, 0, False)  # a ragged last chunk
    forward_case(kind, "f32", rows, chunks * v - 3, chunks * v + 3, 1, True)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_forward_just_below_the_many_rows_kernel(kind):
    for cols in (1000, 5000):
        forward_case(kind, "f32", 32 * sms() - 1, cols, cols, 0, True)


# --- backward: blocks that refill their ring ---------------------------------------------

def backward_inputs(kind, rows, cols, pitch, off):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(rows + 3 * cols + off)
    x = matrix(rows, cols, kind, pitch, off, gen, offset=3.0)
    dy = matrix(rows, cols, kind, pitch, off, gen, scale=False)
    gamma = 1 + 0.1 * torch.randn(cols, device="cuda", generator=gen)
    v = x.double()
    mean = v.mean(1).float()
    rstd = ((v - v.mean(1, keepdim=True)).square_().mean(1) + 1e-5).rsqrt_().float()
    return dy, x, gamma, mean, rstd


def backward_case(kind, rows, cols, pitch, off):
    dy, x, gamma, mean, rstd = backward_inputs(kind, rows, cols, pitch, off)
    out, buf = target(rows, cols, kind, pitch, off)
    dx, dgamma, dbeta = B.layernorm_backward(dy, x, gamma, mean, rstd, out=out)
    d, r = dy.double(), rstd.double()[:, None]
    u = (x.double() - mean.double()[:, None]) * r
    g = d * gamma.double()
    c1, c2 = g.mean(1, keepdim=True), (g * u).mean(1, keepdim=True)
    wx = r * (g - c1 - u * c2)
    # as linear_ref.layernorm_backward
    depth = 64 + cols / 256
    e1 = (depth + 2) * R.U32 * g.abs().mean(1, keepdim=True)
    e2 = (depth + 6) * R.U32 * (g * u).abs_().mean(1, keepdim=True)
    ex = r * (4 * R.U32 * (g.abs() + c1.abs() + (u * c2).abs_()) + e1 + u.abs() * e2 + 2 * R.U32 * u.abs() * c2.abs())
    close(dx, wx, ex, kind)
    # Down a column: a block's rows in one chain (152 blocks or more, so rows / 152 of them), at
    # most 1216 blocks joined in eight chains, those in one.  Two roundings in u, one in its
    # product with dy.
    chain = rows / 152 + 1216 / 8 + 8 + 3
    close(dgamma, (d * u).sum(0), chain * R.U32 * (d * u).abs_().sum(0))
    close(dbeta, d.sum(0), chain * R.U32 * d.abs().sum(0))
    out.fill_(-3.0)
    assert bool((buf == -3.0).all())


def wrapping_rows(cols):
    """Rows that give every block 16 or 17 of them or more (a ring holds 8 at most), with
    some blocks a row short."""
    blocks = sms() * (8 if cols <= 1024 else 4 if cols <= 2048 else 2)
    return blocks * 17 - 50


# Up to 8192 columns a row's values stay in registers between the walks; above, the ring is
# read twice and refilled one stage behind.  fp32 rows over 11568 columns do not fit the ring.
@pytest.mark.parametrize("cols", [300, 1024, 2048, 4096, 7919, 8192, 8193, 9000, 11000, 11568, 11569, 16384])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_backward_goes_round_its_ring(kind, cols):
    v = 8 if kind == "bf16" else 4
    rows = wrapping_rows(cols)
    pitch = -(-cols // v) * v
    backward_case(kind, rows, cols, pitch, 0)
    backward_case(kind, rows, cols, pitch + 1, 3)


@pytest.mark.parametrize("cols", [8192, 11000])
def test_backward_round_its_ring_repeats_bit_for_bit(cols):
    import torch
    args = backward_inputs("bf16", wrapping_rows(cols), cols, cols, 0)
    first = B.layernorm_backward(*args)
    for _ in range(10):
        for a, b in zip(B.layernorm_backward(*args), first):
            assert torch.equal(a, b)
