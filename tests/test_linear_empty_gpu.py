"""The linear layer's conveniences on empty matrices: what they return is written."""
import pytest

from shared_memory_tiled_gb300 import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from shared_memory_tiled_gb300 import build
    build.build()
    B.load()


@pytest.mark.parametrize("on_stream", [False, True])
@pytest.mark.parametrize("kind", ["bfloat16", "float32"])
def test_layernorm_without_columns_has_no_statistics(kind, on_stream):
    """A mean of no values is 0 / 0, and so is its deviation: NaN, not what the memory held."""
    import torch
    dt = getattr(torch, kind)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side if on_stream else torch.cuda.current_stream()):
        held = [torch.full((700,), 7.0, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    del held  # its memory is what the next vectors of 700 get
    y, mean, rstd = B.layernorm(torch.empty(700, 0, dtype=dt, device="cuda"), torch.empty(0, device="cuda"),
                                torch.empty(0, device="cuda"), stream=side.cuda_stream if on_stream else None)
    torch.cuda.synchronize()
    assert y.shape == (700, 0) and mean.shape == rstd.shape == (700,)
    assert bool(mean.isnan().all()) and bool(rstd.isnan().all())
    dx, dgamma, dbeta = B.layernorm_backward(y, y, torch.empty(0, device="cuda"), mean, rstd)
    assert dx.shape == (700, 0) and dgamma.shape == dbeta.shape == (0,)


def test_layernorm_without_rows():
    import torch
    y, mean, rstd = B.layernorm(torch.empty(0, 9, device="cuda"), torch.ones(9, device="cuda"))
    assert y.shape == (0, 9) and mean.shape == rstd.shape == (0,)


def test_quantize_nothing():
    import torch
    for shape in [(0, 300), (300, 0), (0, 0)]:
        q, s, qt, st = B.quantize_fp8(torch.empty(shape, device="cuda"), transposed=True)
        assert q.shape == shape and qt.shape == shape[::-1]
        assert s.numel() == 0 and st.numel() == 0
