"""The 64-bit forms of root-mean-square norm and of the adapters: against differences, and that the check
of 8-bit codes sees a wrong one (no GPU)."""
import numpy as np
import pytest

import linear_ref as R
import norm_ref as N


def test_backward_against_differences():
    rng = np.random.default_rng(1)
    h, gamma, dy, dres = rng.standard_normal((3, 7)), rng.standard_normal(7), rng.standard_normal((3, 7)), rng.standard_normal((3, 7))
    eps, d = 1e-3, 1e-6

    def loss(h, gamma):  # dy reaches y, dres reaches h
        return (N.rmsnorm(h, gamma, eps)[0] * dy).sum() + (h * dres).sum()

    dx, dgamma, _, _ = N.rmsnorm_backward(dy, h, gamma, N.rmsnorm(h, gamma, eps)[1], dres)
    for i in np.ndindex(3, 7):
        e = np.zeros((3, 7))
        e[i] = d
        # central differences: the third derivative times d^2, and 2^-52 of a loss of about 10 over d
        assert abs((loss(h + e, gamma) - loss(h - e, gamma)) / (2 * d) - dx[i]) < 1e-7
    for j in range(7):
        e = np.zeros(7)
        e[j] = d
        assert abs((loss(h, gamma + e) - loss(h, gamma - e)) / (2 * d) - dgamma[j]) < 1e-7


@pytest.mark.parametrize("kind", ["e4m3", "e5m2"])
def test_code_check_sees_a_neighbour(kind):
    rng = np.random.default_rng(2)
    y = rng.standard_normal((4, 200)).astype(np.float32).astype(np.float64)
    codes, scale = R.quantize(y.astype(np.float32), kind, 1)
    N.check_quantized(codes, scale, y, np.abs(y) * 2.0 ** -22, kind)
    for i in ((0, 0), (3, 199)):
        wrong = codes.copy()
        wrong[i] ^= 1
        with pytest.raises(AssertionError):
            N.check_quantized(wrong, scale, y, np.abs(y) * 2.0 ** -22, kind)
    with pytest.raises(AssertionError):
        N.check_quantized(codes, scale * np.float32(1 + 2.0 ** -18), y, np.abs(y) * 2.0 ** -22, kind)


def test_adapters_by_hand():
    x, a, b = np.array([[1.0, 2.0], [3.0, 4.0]]), np.array([[[1.0, -1.0]]]), np.array([[[2.0], [3.0]]])
    out, bound = N.adapters(x, a, b, [0.5], np.array([0, -1]), np.array([[10.0, 20.0], [30.0, 40.0]]))
    assert np.array_equal(out, [[9.0, 18.5], [30.0, 40.0]]) and not bound[1].any()
