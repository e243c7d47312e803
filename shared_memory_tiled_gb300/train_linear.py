"""A linear layer behind a norm, trained and then asked in 8-bit floating point.

    python -m shared_memory_tiled_gb300.train_linear [--steps 60] [--tokens 4096]
                                                      [--inner 1024] [--outer 768]
                                                      [--norm layer|rms] [--requests 0]

The layer learns a teacher of its own shape from synthetic tokens.  One step runs
the operators as a training program does:

    y, mean, rstd = layernorm(x, gamma, beta)
    out = y w^T                       y by rows, w in 128 x 128 blocks
    dw  = dout^T y                    both transposed, contracted over the tokens
    dy  = dout w                      dout by rows, w transposed
    dx, dgamma, dbeta = layernorm_backward(dy, x, gamma, mean, rstd)

Each tensor is quantized once, row by row and transposed from one read, because the
three products contract over three different axes.  Weights and their gradients
stay in fp32.  Afterwards one token is answered from the quantized weight.

With ``--norm rms`` the norm is root-mean-square norm of a residual stream that the input is
added to, and leaves its rows in 8 bits itself; with ``--requests`` that many requests are
answered at once, most with a low-rank adapter of their own beside the shared weight.
"""
from __future__ import annotations

import argparse


class NormedLinear:
    """fp32 parameters of the layer and the operators' calls on them.  ``norm``: "layer", or
    "rms" (no bias, and a residual stream that the input is added to)."""

    def __init__(self, inner: int, outer: int, seed: int = 0, norm: str = "layer"):
        import torch
        if norm not in ("layer", "rms"):
            raise ValueError(f"norm {norm!r}: expected 'layer' or 'rms'")
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.norm = norm
        self.gamma = torch.ones(inner, device="cuda")
        self.beta = torch.zeros(inner, device="cuda") if norm == "layer" else None
        self.w = torch.randn(outer, inner, device="cuda", generator=g) / inner ** 0.5

    def forward(self, x, residual=None):
        """(output, what the backward pass needs); with a residual what is normed is x + residual,
        the first thing that the backward pass needs."""
        from . import binding as B
        if self.norm == "rms":
            yq, ys, yt, yts, h, rstd = B.rmsnorm_fp8(x, self.gamma, residual, transposed=True)
            wq, ws, wt, wts = B.quantize_fp8(self.w, block_rows=128, transposed=True)
            return B.matmul_fp8(yq, ys, wq, ws), (h, None, rstd, yt, yts, wt, wts)
        if residual is not None:
            raise ValueError("a residual goes with norm 'rms'")
        y, mean, rstd = B.layernorm(x, self.gamma, self.beta)
        yq, ys, yt, yts = B.quantize_fp8(y, transposed=True)
        wq, ws, wt, wts = B.quantize_fp8(self.w, block_rows=128, transposed=True)
        return B.matmul_fp8(yq, ys, wq, ws), (x, mean, rstd, yt, yts, wt, wts)

    def backward(self, dout, kept, dresidual=None):
        """(dx, {parameter: gradient}); ``dresidual``: the gradient that reaches the stream past the layer."""
        import torch

        from . import binding as B
        x, mean, rstd, yt, yts, wt, wts = kept
        dq, ds, dt, dts = B.quantize_fp8(dout, dtype=torch.float8_e5m2, transposed=True)
        dw = B.matmul_fp8(dt, dts, yt, yts, out_dtype=torch.float32)
        dy = B.matmul_fp8(dq, ds, wt, wts)
        if self.norm == "rms":
            dx, dgamma = B.rmsnorm_backward(dy, x, self.gamma, rstd, dresidual=dresidual)
            return dx, {"w": dw, "gamma": dgamma}
        if dresidual is not None:
            raise ValueError("a residual's gradient goes with norm 'rms'")
        dx, dgamma, dbeta = B.layernorm_backward(dy, x, self.gamma, mean, rstd)
        return dx, {"w": dw, "gamma": dgamma, "beta": dbeta}

    def answer(self, x, adapters=None):
        """One token's (or a few tokens') output.  ``adapters`` (with norm "rms", x in bf16): (plan, a, b,
        scale), low-rank adapters of the tokens' requests as ``binding.adapters`` takes them."""
        from . import binding as B
        if self.norm == "rms":
            import torch
            rows, inner = x.shape
            y = None
            if adapters is not None:  # they read the rows that are not quantized, on 16-byte boundaries
                y = torch.empty_strided((rows, inner), ((inner + 7) // 8 * 8, 1), dtype=x.dtype, device=x.device)
            q, scale, _, _ = B.rmsnorm_fp8(x, self.gamma, out=y)
            out = B.matmul_fp8(q, scale, *B.quantize_fp8(self.w, block_rows=128))
            if adapters is None:
                return out
            plan, a, b, s = adapters
            return B.adapters(y, a, b, plan, scale=s, base=out, out=out)
        if adapters is not None:
            raise ValueError("adapters go with norm 'rms'")
        y, _, _ = B.layernorm(x, self.gamma, self.beta)
        return B.matmul_fp8(*B.quantize_fp8(y), *B.quantize_fp8(self.w, block_rows=128))


def _normed(x, norm):
    """x, or rows of it, normed in 32 bits."""
    import torch
    x = x.float()
    if norm == "rms":
        return x * torch.rsqrt(x.square().mean(1, keepdim=True) + 1e-6)
    return torch.nn.functional.layer_norm(x, x.shape[1:])


def train(steps: int = 60, tokens: int = 4096, inner: int = 1024, outer: int = 768, rate: float = 0.3,
          norm: str = "layer"):
    """Trains a layer on a teacher's answers; returns (layer, teacher, losses)."""
    import torch
    layer, teacher = NormedLinear(inner, outer, 1, norm), NormedLinear(inner, outer, 2, norm)
    g = torch.Generator(device="cuda").manual_seed(3)
    losses = []
    for _ in range(steps):
        x = torch.randn(tokens, inner, device="cuda", generator=g)
        if norm == "layer":  # which takes the mean out; behind the other one it is a direction along which steps of `rate` diverge
            x.add_(0.5)
        x = x.bfloat16()
        want = _normed(x, norm) @ teacher.w.t()
        out, kept = layer.forward(x)
        off = out.float() - want
        losses.append(off.square().mean())
        _, grads = layer.backward((off / tokens).bfloat16(), kept)
        for name, grad in grads.items():
            getattr(layer, name).sub_(grad, alpha=rate)
    return layer, teacher, [v.item() for v in losses]


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--inner", type=int, default=1024)
    ap.add_argument("--outer", type=int, default=768)
    ap.add_argument("--norm", choices=["layer", "rms"], default="layer")
    ap.add_argument("--requests", type=int, default=0, help="answered at once with adapters (norm rms)")
    a = ap.parse_args()
    if a.requests and a.norm != "rms":
        ap.error("--requests goes with --norm rms")
    import torch
    layer, teacher, losses = train(a.steps, a.tokens, a.inner, a.outer, norm=a.norm)
    for i in range(0, a.steps, max(1, a.steps // 10)):
        print(f"step {i:4d}  loss {losses[i]:.5f}")
    print(f"step {a.steps - 1:4d}  loss {losses[-1]:.5f}")
    x = torch.randn(1, a.inner, device="cuda").bfloat16()
    want = _normed(x, a.norm) @ teacher.w.t()
    got = layer.answer(x).float()
    print(f"one token: {((got - want).norm() / want.norm()).item():.3f} of the teacher's answer off")
    if a.requests:
        off = answer_requests(layer, a.requests)
        print(f"{a.requests} requests, every ninth without an adapter: {off:.3f} of the answers in 32 bits off")


def adapter_of(requests: int, adapters: int, device=None):
    """The adapter of each request: all of them in turn, and none (-1) for every ninth request; two numbers without
    a common factor (8 adapters), so that no adapter goes without a request."""
    import torch
    index = torch.arange(requests, device=device, dtype=torch.int32) % adapters
    index[8::9] = -1
    return index


def answer_requests(layer, requests: int, rank: int = 16, adapters: int = 8) -> float:
    """Answers one token of each request at once, every ninth without an adapter; returns how far
    the answers are from the same in 32 bits (relative norm)."""
    import torch

    from . import binding as B
    outer, inner = layer.w.shape
    g = torch.Generator(device="cuda").manual_seed(5)
    pitch = (inner + 7) // 8 * 8
    a = torch.randn(adapters, rank, pitch, device="cuda", generator=g).div_(inner ** 0.5).bfloat16()[:, :, :inner]
    b = torch.randn(adapters, outer, rank, device="cuda", generator=g).div_(rank ** 0.5).bfloat16()
    scale = torch.rand(adapters, device="cuda", generator=g) + 0.5
    index = adapter_of(requests, adapters, "cuda")
    x = torch.randn(requests, inner, device="cuda", generator=g).bfloat16()
    got = layer.answer(x, (B.adapter_plan(index, adapters), a, b, scale)).float()
    y = _normed(x, "rms") * layer.gamma
    want = y @ layer.w.t()
    for i in range(adapters):
        at = index == i
        want[at] += scale[i] * (y[at] @ a[i].float().t() @ b[i].float().t())
    return ((got - want).norm() / want.norm()).item()


if __name__ == "__main__":
    main()
