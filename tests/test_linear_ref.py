"""The 64-bit forms themselves: 8-bit codes against torch's types on the CPU,
and layer norm's gradients against differences."""
import numpy as np
import pytest

import linear_ref as R


@pytest.mark.parametrize("kind", ["e4m3", "e5m2"])
def test_codes_and_rounding_agree_with_torch(kind):
    import torch
    t8 = torch.float8_e4m3fn if kind == "e4m3" else torch.float8_e5m2
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(t8).to(torch.float64).numpy()
    assert np.array_equal(R.fp8_values(codes.numpy(), kind), want, equal_nan=True)
    rng = np.random.default_rng(0)
    finite = np.sort(want[np.isfinite(want)])
    mid = (finite[1:] + finite[:-1]) / 2            # ties, and their neighbours
    x = np.concatenate([finite, mid, np.nextafter(mid, 1e9), np.nextafter(mid, -1e9),
                        rng.standard_normal(20000) * 100]).astype(np.float32)
    x = x[np.abs(x) <= float(R.TOP[kind])]
    got, ref = R.fp8(x, kind), torch.from_numpy(x).to(t8).view(torch.uint8).numpy()
    assert np.array_equal(got & 0x7F, ref & 0x7F) and np.array_equal(got[x != 0], ref[x != 0])


def test_layernorm_gradients_against_differences():
    rng = np.random.default_rng(1)
    x, dy = rng.standard_normal((5, 37)) + 0.5, rng.standard_normal((5, 37))
    gamma, beta, eps = 1 + 0.1 * rng.standard_normal(37), rng.standard_normal(37), 1e-5

    def loss(x, gamma, beta):
        return (R.layernorm(x, gamma, beta, eps)[0] * dy).sum()

    _, mean, rstd, *_ = R.layernorm(x, gamma, beta, eps)
    dx, dg, db, *_ = R.layernorm_backward(dy, x, gamma, mean, rstd)
    h = 1e-6
    for i, j in [(0, 0), (2, 17), (4, 36)]:
        e = np.zeros_like(x)
        e[i, j] = h
        assert abs((loss(x + e, gamma, beta) - loss(x - e, gamma, beta)) / (2 * h) - dx[i, j]) < 1e-7
    for j in (0, 20, 36):
        e = np.zeros(37)
        e[j] = h
        assert abs((loss(x, gamma + e, beta) - loss(x, gamma - e, beta)) / (2 * h) - dg[j]) < 1e-7
        assert abs((loss(x, gamma, beta + e) - loss(x, gamma, beta - e)) / (2 * h) - db[j]) < 1e-7
