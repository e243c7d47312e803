"""The operators together: the layer of ``train_linear`` against a 32-bit layer, and
that it learns."""
import pytest

from shared_memory_tiled_gb300 import binding as B
from shared_memory_tiled_gb300 import train_linear as T

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from shared_memory_tiled_gb300 import build
    build.build()
    B.load()


def test_one_step_against_32_bits():
    """An e4m3 value is within 2^-4 of what it stands for and an e5m2 value within 2^-3,
    with errors that are as often up as down: a product of thousands of them is off
    by about their root mean square, below 2^-4 and 2^-3 of the result's norm."""
    import torch
    layer = T.NormedLinear(1000, 520, 1)
    layer.gamma = torch.rand(1000, device="cuda") + 0.5
    layer.beta = torch.randn(1000, device="cuda") * 0.1
    x = (torch.randn(3000, 1000, device="cuda") + 0.5).bfloat16()
    dout = torch.randn(3000, 520, device="cuda").bfloat16()
    out, kept = layer.forward(x)
    dx, grads = layer.backward(dout, kept)
    ps = [t.clone().requires_grad_() for t in (x.float(), layer.gamma, layer.beta, layer.w)]
    ref = torch.nn.functional.layer_norm(ps[0], (1000,), ps[1], ps[2]) @ ps[3].t()
    ref.backward(dout.float())

    def off(a, b):
        return ((a.float() - b).norm() / b.norm()).item()

    assert off(out, ref.detach()) < 2 ** -4
    assert off(grads["w"], ps[3].grad) < 2 ** -3
    assert off(grads["gamma"], ps[1].grad) < 2 ** -3
    assert off(grads["beta"], ps[2].grad) < 2 ** -3
    assert off(dx, ps[0].grad) < 2 ** -3
    one = layer.answer(x[:1])
    assert off(one, ref.detach()[:1]) < 2 ** -4


def test_it_learns():
    _, _, losses = T.train(steps=40, tokens=2048, inner=512, outer=300)
    assert losses[-1] < 0.05 * losses[0], losses
