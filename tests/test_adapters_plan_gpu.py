"""A plan of another batch, which only the kernels can tell: nothing is written, and tr_device_status says so."""
from __future__ import annotations

import pytest

from shared_memory_tiled_gb300 import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from shared_memory_tiled_gb300 import build
    build.build()
    B.load()


def call(plan, x, a, b, out):
    tokens, k = x.shape
    adapters, n, rank = b.shape
    B.check(B.tr_adapters(B.AdaptersArgs(
        x=x.data_ptr(), a=a.data_ptr(), b=b.data_ptr(), plan=plan.data_ptr(), out=out.data_ptr(), plan_bytes=plan.numel(),
        out_dtype=B.DType.BF16, tokens=tokens, adapters=adapters, k=k, n=n, rank=rank, ld_x=k, ld_a=k, stride_a=k * rank, ld_b=rank,
        stride_b=n * rank, ld_base=n, ld_out=n)))


def make(index, adapters, room):
    import torch
    plan = torch.zeros(room, dtype=torch.uint8, device="cuda")
    B.check(B.tr_adapter_plan(B.AdapterPlanArgs(index=index.data_ptr(), plan=plan.data_ptr(), plan_bytes=room, tokens=index.numel(),
                                                adapters=adapters)))
    return plan


# one kernel for few tokens, both kernels, the one for many
@pytest.mark.parametrize("tokens", [1, 20, 200, 2100])
def test_a_plan_of_other_sizes(tokens):
    import torch
    x, a = torch.randn(tokens, 64, device="cuda").bfloat16(), torch.randn(3, 16, 64, device="cuda").bfloat16()
    b, room = torch.randn(3, 48, 16, device="cuda").bfloat16(), B.tr_adapter_plan_bytes(tokens + 1, 4)
    index = (torch.arange(tokens + 1, device="cuda") % 3).int()
    good = make(index[:tokens], 3, room)
    want = torch.empty(tokens, 48, dtype=torch.bfloat16, device="cuda")
    call(good, x, a, b, want)
    assert B.tr_device_status() == B.Status.OK
    others = [make(index, 3, room), make(index[:tokens], 4, room), make(index[:tokens], 2, room), torch.zeros_like(good)]
    for plan in others + ([make(index[:tokens - 1], 3, room)] if tokens > 1 else []):
        out = torch.full_like(want, 7)
        call(plan, x, a, b, out)
        assert B.tr_device_status() == B.Status.ERR_UNSUPPORTED
        assert "plan" in B.tr_last_error() and bool((out == 7).all())
        assert B.tr_device_status() == B.Status.OK   # cleared
        call(good, x, a, b, out)
        assert torch.equal(out, want) and B.tr_device_status() == B.Status.OK


def test_beside_a_wait_that_ran_out():
    """Both at once: the wait is named, and both flags are cleared."""
    import torch
    x, a = torch.randn(20, 64, device="cuda").bfloat16(), torch.randn(3, 16, 64, device="cuda").bfloat16()
    b, out = torch.randn(3, 48, 16, device="cuda").bfloat16(), torch.empty(20, 48, dtype=torch.bfloat16, device="cuda")
    call(torch.zeros(1 << 12, dtype=torch.uint8, device="cuda"), x, a, b, out)
    B.check(B.tr_selftest_bounded_wait_in("adapters", 0, 1_000_000))
    assert B.tr_device_status() == B.Status.ERR_TIMEOUT and B.tr_last_error().split(":")[1].split() == ["adapters"]
    assert B.tr_device_status() == B.Status.OK
