"""The fault flags of the norm's and the adapters' kernels, without any fault: a wait that nothing completes runs
out, tr_device_status names the unit and clears its flag, and its kernels run as before."""
import pytest

from shared_memory_tiled_gb300 import binding as B

UNITS = ["transpose", "matmul_fp8", "layernorm_backward", "rmsnorm", "rmsnorm_backward", "adapters"]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from shared_memory_tiled_gb300 import build
    build.build()
    B.load()


def test_refusals():
    assert B.tr_selftest_bounded_wait_in(None, 0, 1000) == B.Status.ERR_NULL
    assert B.tr_selftest_bounded_wait_in("quantize", 0, 1000) == B.Status.ERR_UNSUPPORTED
    for limit in (0, -1, 2_000_000_001):
        assert B.tr_selftest_bounded_wait_in("rmsnorm", 0, limit) == B.Status.ERR_BAD_DIM


@pytest.mark.gpu
@pytest.mark.parametrize("unit", UNITS)
def test_each_units_flag(unit):
    assert B.tr_device_status() == B.Status.OK
    B.check(B.tr_selftest_bounded_wait_in(unit, 0, 5_000_000))
    assert B.tr_device_status() == B.Status.ERR_TIMEOUT
    assert B.tr_last_error().split(":")[1].split() == [unit]
    B.check(B.tr_selftest_bounded_wait_in(unit, 1, 50_000_000))
    assert B.tr_device_status() == B.Status.OK


@pytest.mark.gpu
def test_the_kernels_run_as_before_afterwards():
    import torch
    x, gamma = torch.randn(400, 1000, device="cuda"), torch.ones(1000, device="cuda")

    def step():
        y, h, rstd = B.rmsnorm(x, gamma, x)
        return [y, h, rstd, *B.rmsnorm_backward(y, h, gamma, rstd, dresidual=x)]

    want = step()
    for unit in UNITS:
        B.check(B.tr_selftest_bounded_wait_in(unit, 0, 1_000_000))
    assert B.tr_device_status() == B.Status.ERR_TIMEOUT
    for a, b in zip(step(), want):
        assert torch.equal(a, b)
    assert B.tr_device_status() == B.Status.OK
