"""The training program at its own sizes and rate, behind either norm: its steps stay finite."""
import math

import pytest

from shared_memory_tiled_gb300 import binding as B
from shared_memory_tiled_gb300 import train_linear as T

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from shared_memory_tiled_gb300 import build
    build.build()
    B.load()


@pytest.mark.parametrize("norm", ["layer", "rms"])
def test_losses_and_weights_stay_finite(norm):
    layer, _, losses = T.train(norm=norm)
    assert len(losses) == 60 and all(math.isfinite(v) for v in losses)
    assert bool(layer.w.isfinite().all()) and bool(layer.gamma.isfinite().all())
