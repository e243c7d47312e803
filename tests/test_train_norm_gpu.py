"""The operators together: the layer of ``train_linear`` behind root-mean-square norm of a residual stream
against a 32-bit layer, answers with adapters, and the command."""
import sys

import pytest

from shared_memory_tiled_gb300 import binding as B
from shared_memory_tiled_gb300 import train_linear as T

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from shared_memory_tiled_gb300 import build
    build.build()
    B.load()


def off(a, b):
    return ((a.float() - b).norm() / b.norm()).item()


@pytest.mark.parametrize("add", [True, False])
def test_one_step_against_32_bits(add):
    """An e4m3 value is within 2^-4 of what it stands for and an e5m2 value within 2^-3, with errors that are as
    often up as down: a product of thousands of them is off by about their root mean square, below 2^-4 and
    2^-3 of the result's norm."""
    import torch
    layer = T.NormedLinear(1000, 520, 1, "rms")
    layer.gamma = torch.rand(1000, device="cuda") + 0.5
    x, res = (torch.randn(3000, 1000, device="cuda").bfloat16() for _ in range(2))
    res = res if add else None
    dout, dres = torch.randn(3000, 520, device="cuda").bfloat16(), torch.randn(3000, 1000, device="cuda").bfloat16()
    out, kept = layer.forward(x, res)
    dx, grads = layer.backward(dout, kept, dresidual=dres if add else None)
    h = x if res is None else (x.float() + res.float()).bfloat16()
    assert torch.equal(kept[0], h)
    ps = [t.clone().requires_grad_() for t in (h.float(), layer.gamma, layer.w)]
    ref = ps[0] * torch.rsqrt(ps[0].square().mean(1, keepdim=True) + 1e-6) * ps[1] @ ps[2].t()
    torch.autograd.backward([ref] + [ps[0]] * add, [dout.float()] + [dres.float()] * add)
    assert off(out, ref.detach()) < 2 ** -4
    assert off(grads["w"], ps[2].grad) < 2 ** -3
    assert off(grads["gamma"], ps[1].grad) < 2 ** -3
    assert off(dx, ps[0].grad) < 2 ** -3
    assert off(layer.answer(h[:1]), ref.detach()[:1]) < 2 ** -4


@pytest.mark.parametrize("requests", [1, 9, 40, 500, 3000])
def test_answers_with_adapters(requests):
    assert T.answer_requests(T.NormedLinear(1000, 520, 1, "rms"), requests) < 2 ** -4


def test_a_captured_decode_step():
    """Norm, product, plan and adapters of one step captured and replayed on new tokens and requests."""
    import torch
    layer = T.NormedLinear(512, 264, 3, "rms")
    a, b = torch.randn(4, 16, 512, device="cuda").bfloat16() / 32, torch.randn(4, 264, 16, device="cuda").bfloat16() / 4
    x, index = torch.randn(24, 512, device="cuda").bfloat16(), torch.randint(-1, 4, (24,), device="cuda", dtype=torch.int32)

    def step():
        return layer.answer(x, (B.adapter_plan(index, 4), a, b, None))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(3):
        x.normal_()
        index.copy_(torch.randint(-1, 4, (24,), device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, step())


def test_the_command_runs(monkeypatch, capsys):
    monkeypatch.setattr(sys, "argv", ["train_linear", "--steps", "2", "--tokens", "512", "--inner", "264", "--outer", "100", "--norm", "rms",
                                      "--requests", "20"])
    T.main()
    assert "20 requests" in capsys.readouterr().out


def test_refusals():
    import torch
    with pytest.raises(ValueError):
        T.NormedLinear(8, 8, norm="group")
    layer, x = T.NormedLinear(64, 8), torch.randn(4, 64, device="cuda")
    with pytest.raises(ValueError):
        layer.forward(x, x)
    with pytest.raises(ValueError):
        layer.answer(x, (None,) * 4)
    out, kept = layer.forward(x)
    with pytest.raises(ValueError):
        layer.backward(out, kept, dresidual=x)
