"""The product where two scales multiplied leave the range of 32 bits and the result does
not: the scales of large values times small codes, and of values far below one."""
from __future__ import annotations

import numpy as np
import pytest

import linear_ref as R
from shared_memory_tiled_gb300 import binding as B
from test_linear_gpu import close, host, torch_types

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from shared_memory_tiled_gb300 import build
    build.build()
    B.load()


def operand(rows, k, block, codes, exponent, seed):
    """Codes drawn from a list, a row of zeros, and scales of one to two times 2^exponent."""
    import torch
    rng = np.random.default_rng(seed)
    q = rng.choice(np.array(codes, np.uint8), (rows, k))
    q[rows // 2] = 0
    s = np.ldexp(1 + rng.random((-(-k // 128), -(-rows // block))), exponent).astype(np.float32)
    held = torch.zeros(rows, -(-k // 16) * 16, dtype=torch.uint8, device="cuda")
    held[:, :k] = torch.from_numpy(q)
    return held.view(torch_types("e4m3"))[:, :k], torch.from_numpy(s).cuda(), q, s


SMALL = [0x00, 0x01, 0x02, 0x81, 0x82]                       # 0, 2^-9, 2^-8 and their negatives
WIDE = [0x00, 0x38, 0x45, 0x60, 0x7E, 0xB8, 0xC9, 0xFE]      # 1 to 448


@pytest.mark.parametrize("ab,bb", [(1, 1), (1, 128), (128, 1), (128, 128)])
@pytest.mark.parametrize("m,n,k", [(3, 200, 300), (40, 129, 1000), (150, 333, 700), (2304, 2304, 300)])
@pytest.mark.parametrize("codes,ea,eb", [(SMALL, 70, 60), (SMALL, 20, 110), (WIDE, -75, -60), (WIDE, -30, -110)])
def test_scales_whose_product_leaves_the_range(codes, ea, eb, m, n, k, ab, bb):
    """Sums of k products of 2^-16 at most times 2^132 and of 2^18 times 2^-138: both
    are normal numbers in 32 bits."""
    import torch
    a, sa, qa, ha = operand(m, k, ab, codes, ea, m + ab)
    b, sb, qb, hb = operand(n, k, bb, codes, eb, n + bb)
    want, bound = R.matmul(qa, ha, "e4m3", ab, qb, hb, "e4m3", bb)
    # a sum may come out below the normal numbers by cancellation; a rounding there is 2^-150
    close(host(B.matmul_fp8(a, sa, b, sb, out_dtype=torch.float32)), want, bound + 2.0 ** -149)


def test_one_block_out_of_range_leaves_the_others_as_they_are():
    """Rows whose scales are ordinary give the same bits beside rows that are not."""
    import torch
    for m, n in [(40, 200), (200, 200), (2304, 2304)]:
        for bb in (1, 128):
            a, sa, qa, ha = operand(m, 400, 1, WIDE, -8, 1)
            b, sb, qb, hb = operand(n, 400, bb, WIDE, -8, 2)
            first = B.matmul_fp8(a, sa, b, sb, out_dtype=torch.float32)
            sa[1, 7::9] = 2.0 ** 125
            sa[2, 3::9] = 2.0 ** -125
            got = B.matmul_fp8(a, sa, b, sb, out_dtype=torch.float32)
            same = torch.ones(m, dtype=torch.bool)
            same[7::9] = same[3::9] = False
            assert torch.equal(got[same.cuda()], first[same.cuda()])


@pytest.mark.parametrize("m,n", [(3, 200), (40, 129), (150, 333), (2304, 2304)])
@pytest.mark.parametrize("bb", [1, 128])
def test_masked_rows_are_zero_and_the_others_right(m, n, bb):
    """Rows and blocks of zeros as the quantizer leaves them, in e5m2: their scale times a
    weight's is below the normal numbers."""
    import torch
    k = 1000
    rng = np.random.default_rng(m)
    x = rng.standard_normal((m, k)).astype(np.float32)
    x[rng.random(m) < 0.3] = 0
    x[1, 128:256] = 0
    w = (0.01 * rng.standard_normal((n, k))).astype(np.float32)
    w[:, 256:384] = 0
    a, sa = B.quantize_fp8(torch.from_numpy(x).cuda(), dtype=torch.float8_e5m2)
    b, sb = B.quantize_fp8(torch.from_numpy(w).cuda(), block_rows=bb)
    qa, ha = R.quantize(x, "e5m2", 1)
    qb, hb = R.quantize(w, "e4m3", bb)
    want, bound = R.matmul(qa, ha, "e5m2", 1, qb, hb, "e4m3", bb)
    got = host(B.matmul_fp8(a, sa, b, sb, out_dtype=torch.float32))
    close(got, want, bound)
    assert not got[(x == 0).all(1)].any()


@pytest.mark.parametrize("m,n", [(40, 129), (150, 333), (2304, 2304)])
def test_scales_of_every_size_in_one_tile(m, n):
    """Each row and column with an exponent of its own, so that products of scales run from
    2^-170 to 2^171 in one block: whatever is finite is right, down to the spacing of the
    subnormal numbers."""
    import torch
    for codes in (SMALL, WIDE):
        a, sa, qa, ha = operand(m, 128, 1, codes, 0, m)
        b, sb, qb, hb = operand(n, 128, 1, codes, 0, n + 1)
        rng = np.random.default_rng(5)
        ha = np.ldexp(ha, rng.integers(-85, 86, ha.shape)).astype(np.float32)
        hb = np.ldexp(hb, rng.integers(-85, 86, hb.shape)).astype(np.float32)
        want, bound = R.matmul(qa, ha, "e4m3", 1, qb, hb, "e4m3", 1)
        got = host(B.matmul_fp8(a, torch.from_numpy(ha).cuda(), b, torch.from_numpy(hb).cuda(), out_dtype=torch.float32))
        finite = np.abs(want) + bound < 2.0 ** 127
        close(got[finite], want[finite], bound[finite] + 2.0 ** -148)
        assert not np.isnan(got).any()
