"""The adapters on inputs whose outputs are known to the last bit (``adapter_exact``): through rings that go round many
times, for each width of the inner values, outputs on and off 16-byte boundaries.  Without a GPU: that the check sees what it is for."""
from __future__ import annotations

import numpy as np
import pytest

import adapter_exact as E
from shared_memory_tiled_gb300 import binding as B


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from shared_memory_tiled_gb300 import build
    build.build()
    B.load()


# --- the check itself ----------------------------------------------------------------------

def test_terms_stand_for_their_value():
    rng = np.random.default_rng(1)
    v = (rng.standard_normal(200000) * np.exp(5 * rng.standard_normal(200000))).astype(np.float32)
    wide = v.astype(np.float64)
    two, three = E.terms(v, 2), E.terms(v, 3)
    assert np.array_equal(sum(t.astype(np.float64) for t in three), wide)
    off = np.abs(sum(t.astype(np.float64) for t in two) / wide - 1)
    assert off.max() <= 2.0 ** -16 and off.max() > 2.0 ** -17
    for t in two + three:   # in bf16, of the value's sign, never zero, and no larger
        assert np.array_equal(E.bf16(t)[0], t) and np.all(t * np.sign(v) > 0) and np.all(np.abs(t) <= np.abs(v))
    v = E.bf16(v)[0]        # nothing left after the first
    for count in (2, 3):
        got = E.terms(v, count)
        assert np.array_equal(sum(got), v) and all(np.all(t * np.sign(v) > 0) for t in got)
        assert all(not t.any() for t in E.terms(np.zeros(3, np.float32), count))
        for special in (np.inf, -np.inf, np.nan):
            assert all(np.array_equal(t, [special], equal_nan=True) for t in E.terms(np.array([special], np.float32), count))


def emulated(x, a, b, scale, index, base, count, k_less=None, lost=0):
    """The formula in 64 bits with `count` terms to an inner value, the last `lost` left out; `k_less`: 64 values of k left out."""
    x, out = x.astype(np.float64), np.zeros((x.shape[0], b.shape[1])) + (0 if base is None else base)
    if k_less is not None:
        x = x.copy()
        x[:, k_less:k_less + 64] = 0
    for g in range(a.shape[0]):
        at = index == g
        v = (x[at] @ a[g].T.astype(np.float64)).astype(np.float32) * scale[g]
        out[at] += sum(t.astype(np.float64) for t in E.terms(v, count)[:count - lost]) @ b[g].T.astype(np.float64)
    return out


def test_the_checks_see_a_lost_term_and_a_lost_piece():
    for k, rank in ((520, 16), (4096, 64), (8192, 24), (2048, 128)):
        x, a, b, scale, base, index = E.whole(40, 3, k, 24, rank, k)
        right = emulated(x, a, b, scale, index, base, 2)
        assert np.array_equal(right, emulated(x, a, b, scale, index, base, 3))      # two terms hold them
        assert np.array_equal(right, right.astype(np.float32))
        for less in (0, k - 64):
            wrong = emulated(x, a, b, scale, index, base, 2, less)
            assert (wrong[index >= 0] != right[index >= 0]).mean() > 0.5, (k, less)
        x, a, b, scale, index = E.single(40, 3, k, 200, rank, k)
        right = emulated(x, a, b, scale, index, None, 3)
        assert np.array_equal(right, right.astype(np.float32))
        less = emulated(x, a, b, scale, index, None, 3, lost=1)                    # fp32 outputs: equality
        assert (less[index >= 0] != right[index >= 0]).mean() > 0.3
        two, one = (E.bf16(emulated(x, a, b, scale, index, None, 2, lost=n))[0].astype(np.float64) for n in (0, 1))
        assert np.all(np.abs(two - right) <= E.BITS["bf16"] * np.abs(right))
        assert (np.abs(one - right) > E.BITS["bf16"] * np.abs(right)).sum() > 100


# --- the kernels ---------------------------------------------------------------------------

def on_gpu(v):
    """bf16 rows on 16-byte boundaries."""
    import torch
    t = torch.zeros(*v.shape[:-1], -(-v.shape[-1] // 8) * 8, dtype=torch.bfloat16, device="cuda")[..., :v.shape[-1]]
    return t.copy_(torch.from_numpy(v).cuda())


def wide(x, a, b, scale, index, base):
    import torch
    out = torch.zeros(x.shape[0], b.shape[1], dtype=torch.float64, device="cuda") if base is None else base.double()
    for g in range(a.shape[0]):
        at = torch.nonzero(index == g)[:, 0]
        v = (x[at].double() @ a[g].double().t()).float() * scale[g]
        assert not at.numel() or base is None or (v.abs() @ b[g].float().abs().t()).max().item() < 2 ** 21
        out[at] += v.double() @ b[g].double().t()
    return out


def answers(case, out, seed):
    """(whole: output and what it has to be, single: the same)"""
    import torch
    from test_linear_gpu import torch_types
    x, a, b, scale, base, index = E.whole(*case, seed)
    x, a, b, scale = on_gpu(x), on_gpu(a), on_gpu(b), torch.from_numpy(scale).cuda()
    index, base = torch.from_numpy(index).cuda(), torch.from_numpy(base).cuda().to(torch_types(out))
    got = B.adapters(x, a, b, B.adapter_plan(index, case[1]), scale=scale, base=base)
    want = wide(x, a, b, scale, index, base)
    x, a, b, scale, index = E.single(*case, seed)
    x, a, b, scale, index = on_gpu(x), on_gpu(a), on_gpu(b), torch.from_numpy(scale).cuda(), torch.from_numpy(index).cuda()
    alone = B.adapters(x, a, b, B.adapter_plan(index, case[1]), scale=scale, out_dtype=torch_types(out))
    return got, want, alone, wide(x, a, b, scale, index, None)


# tokens, adapters, k, n, rank: in k_adapters a CTA's chunks of k go round its ring twice and more, for each width of the
# inner values, alone in its cluster and not, and its tiles of columns round b's ring and the slots of base; odd sizes; some
# tiles of both kernels side by side; few tokens of long rows
CASES = [(6000, 3, 4096, 2048, 16), (6000, 3, 4096, 2049, 12), (6000, 3, 4095, 2048, 32), (6000, 3, 4096, 2050, 24), (6000, 3, 4096, 2048, 64),
         (6000, 3, 4090, 2047, 48), (6000, 3, 2048, 2048, 128), (6000, 3, 2048, 2041, 100), (20000, 2, 2048, 1032, 16), (20000, 2, 2048, 1031, 64),
         (2500, 4, 8192, 4104, 24), (2500, 4, 8190, 4099, 16), (1900, 5, 8192, 2056, 24), (1900, 5, 8192, 2055, 16), (500, 20, 4096, 1032, 64),
         (1, 2, 8192, 1032, 16), (9, 3, 8192, 1031, 24), (30, 4, 4096, 520, 64), (64, 40, 8192, 2048, 16), (32, 3, 2048, 2041, 128), (64, 2, 8191, 264, 16)]


@pytest.mark.gpu
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("case", CASES)
def test_to_the_last_bit(case, out):
    import torch
    got, want, alone, single = answers(case, out, sum(case))
    assert torch.equal(got, want.to(got.dtype))
    if out == "f32":
        assert torch.equal(alone.double(), single)
    else:
        assert bool(((alone.double() - single).abs() <= E.BITS[out] * single.abs()).all())
    assert B.tr_device_status() == B.Status.OK


@pytest.mark.gpu
def test_a_batch_of_long_prompts():
    """8192 tokens of 8192 values into 8192 columns, rank 64 (inner values and sums as above)."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(1)
    x, a, b = (torch.randint(-1, 2, s, device="cuda", generator=g).bfloat16() for s in ((8192, 8192), (8, 64, 8192), (8, 8192, 64)))
    base = torch.randint(-9, 10, (8192, 8192), device="cuda", generator=g).bfloat16()
    index = torch.from_numpy(E.groups(8192, 8, np.random.default_rng(2))).cuda()
    scale = torch.ones(8, device="cuda")
    got = B.adapters(x, a, b, B.adapter_plan(index, 8), scale=scale, base=base)
    assert torch.equal(got, wide(x, a, b, scale, index, base).to(got.dtype))
    inside = base.clone()
    assert torch.equal(B.adapters(x, a, b, B.adapter_plan(index, 8), base=inside, out=inside), got)
