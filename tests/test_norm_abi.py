"""Root-mean-square norm and the adapters on the host: every argument error comes back
before any CUDA call (no GPU needed; the addresses are never dereferenced)."""
from __future__ import annotations

import ctypes

import pytest

from shared_memory_tiled_gb300 import binding as B
from shared_memory_tiled_gb300 import build as build_mod

S = B.Status
AT = [0x7F0000000000 + i * 0x10000000000 for i in range(12)]  # far apart


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build_mod.build()
    B.load()


def call(f, a, kw):
    for k, v in kw.items():
        setattr(a, k, v)
    return f(a)


def rmsnorm(**kw):
    return call(B.tr_rmsnorm, B.RmsnormArgs(
        x=AT[0], residual=AT[1], gamma=AT[2], h=AT[3], y=AT[4], rstd=AT[5], q=AT[6], scale=AT[7], qt=AT[8], scale_t=AT[9],
        x_dtype=B.DType.BF16, w_dtype=B.DType.F32, q_dtype=B.DType.E4M3, rows=300, cols=500, ld_x=500, ld_residual=500, ld_h=501,
        ld_y=500, ld_q=512, ld_scale=300, ld_qt=304, ld_scale_t=500, eps=1e-6), kw)


def test_rmsnorm_refusals():
    assert B.tr_rmsnorm(None) == S.ERR_NULL
    for bad in (dict(x_dtype=2), dict(w_dtype=3), dict(reserved=1), dict(reserved2=-1), dict(q_dtype=0), dict(q_dtype=7)):
        assert rmsnorm(**bad) == S.ERR_UNSUPPORTED, bad
    for bad in (dict(rows=-1), dict(cols=-1), dict(eps=-1e-9), dict(eps=float("nan")), dict(eps=float("inf"))):
        assert rmsnorm(**bad) == S.ERR_BAD_DIM, bad
    for name in ("x", "gamma", "h", "scale", "scale_t", "rstd", "q"):  # with qt the last two are wanted
        assert rmsnorm(**{name: 0}) == S.ERR_NULL, name
    assert rmsnorm(residual=0) == S.ERR_UNSUPPORTED and "without a residual" in B.tr_last_error()
    for bad in (dict(ld_x=499), dict(ld_residual=499), dict(ld_h=499), dict(ld_y=499), dict(ld_q=496), dict(ld_scale=299),
                dict(ld_qt=288), dict(ld_scale_t=499)):
        assert rmsnorm(**bad) == S.ERR_BAD_LD, bad
    for bad in (dict(x=AT[0] + 1), dict(residual=AT[1] + 1), dict(gamma=AT[2] + 2), dict(h=AT[3] + 1), dict(y=AT[4] + 1),
                dict(rstd=AT[5] + 2), dict(q=AT[6] + 8), dict(scale=AT[7] + 1), dict(qt=AT[8] + 4), dict(scale_t=AT[9] + 2),
                dict(ld_q=520), dict(ld_qt=312)):
        assert rmsnorm(**bad) == S.ERR_UNSUPPORTED, bad
    for bad in (dict(y=AT[0]), dict(h=AT[0]), dict(y=AT[1]), dict(y=AT[3]), dict(q=AT[4]), dict(rstd=AT[2]), dict(qt=AT[6]),
                dict(scale=AT[9]), dict(h=AT[1]),                 # the residual with another pitch
                dict(h=AT[1] + 2, ld_h=500), dict(residual=AT[0], h=AT[0], ld_h=500), dict(residual=AT[3], ld_residual=501, y=AT[3])):
        assert rmsnorm(**bad) == S.ERR_OVERLAP, bad
    assert rmsnorm(rows=1 << 40, ld_x=1 << 40, cols=1 << 40) == S.ERR_BAD_DIM
    assert rmsnorm(rows=0, x=0, h=0) == S.OK and rmsnorm(cols=0, x=0, gamma=0) == S.OK


def backward(**kw):
    return call(B.tr_rmsnorm_backward, B.RmsnormBackwardArgs(
        dy=AT[0], h=AT[1], gamma=AT[2], rstd=AT[3], dresidual=AT[4], dx=AT[5], dgamma=AT[6], workspace=AT[7], workspace_bytes=1 << 20,
        x_dtype=B.DType.BF16, w_dtype=B.DType.F32, rows=20, cols=30, ld_dy=30, ld_h=30, ld_dresidual=30, ld_dx=31), kw)


def test_rmsnorm_backward_refusals():
    assert B.tr_rmsnorm_backward(None) == S.ERR_NULL
    for bad in (dict(x_dtype=2), dict(w_dtype=9)):
        assert backward(**bad) == S.ERR_UNSUPPORTED, bad
    assert backward(rows=-1) == S.ERR_BAD_DIM and backward(cols=-1) == S.ERR_BAD_DIM
    for name in ("dy", "h", "gamma", "rstd", "dx", "dgamma", "workspace"):
        assert backward(**{name: 0}) == S.ERR_NULL, name
    for bad in (dict(ld_dy=29), dict(ld_h=29), dict(ld_dresidual=29), dict(ld_dx=29)):
        assert backward(**bad) == S.ERR_BAD_LD, bad
    need = B.tr_rmsnorm_backward_workspace(20, 30)
    for bad in (dict(workspace_bytes=need - 1), dict(workspace=AT[7] + 8), dict(dgamma=AT[6] + 2), dict(dx=AT[5] + 1), dict(rstd=AT[3] + 2)):
        assert backward(**bad) == S.ERR_UNSUPPORTED, bad
    for bad in (dict(dx=AT[0]), dict(dx=AT[1]), dict(dgamma=AT[2]), dict(workspace=AT[5]), dict(workspace=AT[3]),
                dict(dx=AT[4]), dict(dx=AT[4] + 2, ld_dx=30)):  # dresidual with another pitch, or another place
        assert backward(**bad) == S.ERR_OVERLAP, bad
    assert backward(cols=0, dgamma=0) == S.OK
    assert B.tr_rmsnorm_backward_workspace(-1, 3) == -1 and B.tr_rmsnorm_backward_workspace(3, 1 << 62) == -1
    assert B.tr_rmsnorm_backward_workspace(0, 3) == B.tr_rmsnorm_backward_workspace(3, 0) == 0


def plan(**kw):
    return call(B.tr_adapter_plan, B.AdapterPlanArgs(index=AT[0], plan=AT[1], plan_bytes=1 << 20, tokens=100, adapters=8), kw)


def test_plan_refusals():
    assert B.tr_adapter_plan(None) == S.ERR_NULL
    assert plan(tokens=-1) == S.ERR_BAD_DIM and plan(adapters=-1) == S.ERR_BAD_DIM
    assert plan(index=0) == S.ERR_NULL and plan(plan=0) == S.ERR_NULL
    need = B.tr_adapter_plan_bytes(100, 8)
    for bad in (dict(tokens=1 << 31, plan_bytes=1 << 40), dict(adapters=1 << 15), dict(plan_bytes=need - 1), dict(plan=AT[1] + 8),
                dict(index=AT[0] + 1)):
        assert plan(**bad) == S.ERR_UNSUPPORTED, bad
    assert plan(index=AT[1] + need - 4) == S.ERR_OVERLAP
    assert plan(tokens=0, index=0, plan=0) == S.OK
    assert B.tr_adapter_plan_bytes(1 << 31, 1) == B.tr_adapter_plan_bytes(1, 1 << 15) == B.tr_adapter_plan_bytes(-1, 1) == -1


def adapters(**kw):
    return call(B.tr_adapters, B.AdaptersArgs(
        x=AT[0], a=AT[1], b=AT[2], scale=AT[3], plan=AT[4], base=AT[5], out=AT[6], plan_bytes=1 << 20, out_dtype=B.DType.BF16, tokens=100,
        adapters=8, k=500, n=300, rank=12, ld_x=504, ld_a=504, stride_a=504 * 12, ld_b=16, stride_b=16 * 300, ld_base=300, ld_out=301), kw)


def test_adapters_refusals():
    assert B.tr_adapters(None) == S.ERR_NULL
    for bad in (dict(out_dtype=2), dict(reserved=1), dict(rank=0), dict(rank=129), dict(rank=-1), dict(k=1 << 30), dict(n=1 << 30),
                dict(tokens=1 << 31), dict(adapters=1 << 15)):
        assert adapters(**bad) == S.ERR_UNSUPPORTED, bad
    for name in ("tokens", "adapters", "k", "n"):
        assert adapters(**{name: -1}) == S.ERR_BAD_DIM, name
    for name in ("x", "a", "b", "plan", "out"):
        assert adapters(**{name: 0}) == S.ERR_NULL, name
    for bad in (dict(ld_x=496), dict(ld_a=496), dict(ld_b=8), dict(ld_base=299), dict(ld_out=299), dict(stride_a=504 * 11), dict(stride_b=-8),
                dict(stride_b=16 * 299)):
        assert adapters(**bad) == S.ERR_BAD_LD, bad
    for bad in (dict(x=AT[0] + 2), dict(a=AT[1] + 8), dict(b=AT[2] + 4), dict(scale=AT[3] + 2), dict(plan=AT[4] + 4), dict(base=AT[5] + 1),
                dict(out=AT[6] + 1), dict(ld_x=500), dict(ld_a=501, stride_a=8 * 800), dict(ld_b=12), dict(stride_a=504 * 12 + 4),
                dict(plan_bytes=B.tr_adapter_plan_bytes(100, 8) - 1)):
        assert adapters(**bad) == S.ERR_UNSUPPORTED, bad
    for bad in (dict(out=AT[0]), dict(out=AT[1] + 2 * 504 * 12 * 7), dict(out=AT[2]), dict(out=AT[3]), dict(out=AT[4]), dict(out=AT[5]),
                dict(out=AT[5] + 2, ld_out=300)):
        assert adapters(**bad) == S.ERR_OVERLAP, bad
    assert adapters(tokens=0, x=0, out=0, plan=0) == S.OK and adapters(n=0, b=0, out=0) == S.OK


@pytest.mark.parametrize("pack,struct", [(B._PACK_RMSNORM, B.RmsnormArgs), (B._PACK_RMSNORM_BACKWARD, B.RmsnormBackwardArgs),
                                         (B._PACK_PLAN, B.AdapterPlanArgs), (B._PACK_ADAPTERS, B.AdaptersArgs)])
def test_packed_arguments_are_the_structs(pack, struct):
    values = [i + 1.5 if kind is ctypes.c_float else 1 << (20 + i) if ctypes.sizeof(kind) == 8 else i + 1
              for i, (_, kind) in enumerate(struct._fields_)]
    packed = pack(*values)
    assert len(packed) == ctypes.sizeof(struct)
    held = struct.from_buffer_copy(packed)
    for (name, _), v in zip(struct._fields_, values):
        assert getattr(held, name) == v, name
