"""The fault flags of the product and of layer norm's backward pass, without any fault:
a wait of each unit that nothing completes runs out, and tr_device_status reads and
clears every unit's flag."""
import pytest

from shared_memory_tiled_gb300 import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from shared_memory_tiled_gb300 import build
    build.build()
    B.load()
    assert B.tr_device_status() == B.Status.OK


def test_each_units_flag_is_read_and_cleared():
    B.check(B.tr_selftest_bounded_wait(0, 10_000_000))  # 10 ms each
    assert B.tr_device_status() == B.Status.ERR_TIMEOUT
    units = B.tr_last_error().split(":")[1].split()
    assert units == ["transpose", "matmul_fp8", "layernorm_backward"]
    assert B.tr_device_status() == B.Status.OK


def test_waits_that_complete_raise_none():
    B.check(B.tr_selftest_bounded_wait(1, 50_000_000))
    assert B.tr_device_status() == B.Status.OK


def test_the_units_kernels_run_as_before_afterwards():
    import torch
    B.check(B.tr_selftest_bounded_wait(0, 1_000_000))
    assert B.tr_device_status() == B.Status.ERR_TIMEOUT
    x = torch.randn(300, 256, device="cuda")
    gamma = torch.ones(256, device="cuda")
    y, mean, rstd = B.layernorm(x, gamma)
    want = B.layernorm_backward(y, x, gamma, mean, rstd)
    q, s = B.quantize_fp8(x)
    out = B.matmul_fp8(q, s, q, s, out_dtype=torch.float32)
    assert B.tr_device_status() == B.Status.OK
    v = q.float() * s.t().repeat_interleave(128, 1)
    assert torch.allclose(out, v @ v.t(), rtol=1e-3, atol=1e-3)
    for a, b in zip(B.layernorm_backward(y, x, gamma, mean, rstd), want):
        assert torch.equal(a, b)
