"""A linear layer behind a layer norm, trained and then asked in 8-bit floating point.

    python -m shared_memory_tiled_gb300.train_linear [--steps 60] [--tokens 4096]
                                                      [--inner 1024] [--outer 768]

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
"""
from __future__ import annotations

import argparse


class NormedLinear:
    """fp32 parameters of the layer and the operators' calls on them."""

    def __init__(self, inner: int, outer: int, seed: int = 0):
        import torch
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.gamma = torch.ones(inner, device="cuda")
        self.beta = torch.zeros(inner, device="cuda")
        self.w = torch.randn(outer, inner, device="cuda", generator=g) / inner ** 0.5

    def forward(self, x):
        """(output, what the backward pass needs)"""
        from . import binding as B
        y, mean, rstd = B.layernorm(x, self.gamma, self.beta)
        yq, ys, yt, yts = B.quantize_fp8(y, transposed=True)
        wq, ws, wt, wts = B.quantize_fp8(self.w, block_rows=128, transposed=True)
        return B.matmul_fp8(yq, ys, wq, ws), (x, mean, rstd, yt, yts, wt, wts)

    def backward(self, dout, kept):
        """(dx, {parameter: gradient})"""
        import torch

        from . import binding as B
        x, mean, rstd, yt, yts, wt, wts = kept
        dq, ds, dt, dts = B.quantize_fp8(dout, dtype=torch.float8_e5m2, transposed=True)
        dw = B.matmul_fp8(dt, dts, yt, yts, out_dtype=torch.float32)
        dy = B.matmul_fp8(dq, ds, wt, wts)
        dx, dgamma, dbeta = B.layernorm_backward(dy, x, self.gamma, mean, rstd)
        return dx, {"w": dw, "gamma": dgamma, "beta": dbeta}

    def answer(self, x):
        """One token's (or a few tokens') output."""
        from . import binding as B
        y, _, _ = B.layernorm(x, self.gamma, self.beta)
        return B.matmul_fp8(*B.quantize_fp8(y), *B.quantize_fp8(self.w, block_rows=128))


def train(steps: int = 60, tokens: int = 4096, inner: int = 1024, outer: int = 768, rate: float = 0.3):
    """Trains a layer on a teacher's answers; returns (layer, teacher, losses)."""
    import torch
    layer, teacher = NormedLinear(inner, outer, 1), NormedLinear(inner, outer, 2)
    g = torch.Generator(device="cuda").manual_seed(3)
    losses = []
    for _ in range(steps):
        x = torch.randn(tokens, inner, device="cuda", generator=g).add_(0.5).bfloat16()
        want = torch.nn.functional.layer_norm(x.float(), (inner,)) @ teacher.w.t()
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
    a = ap.parse_args()
    import torch
    layer, teacher, losses = train(a.steps, a.tokens, a.inner, a.outer)
    for i in range(0, a.steps, max(1, a.steps // 10)):
        print(f"step {i:4d}  loss {losses[i]:.5f}")
    print(f"step {a.steps - 1:4d}  loss {losses[-1]:.5f}")
    x = torch.randn(1, a.inner, device="cuda").bfloat16()
    want = torch.nn.functional.layer_norm(x.float(), (a.inner,)) @ teacher.w.t()
    got = layer.answer(x).float()
    print(f"one token: {((got - want).norm() / want.norm()).item():.3f} of the teacher's answer off")


if __name__ == "__main__":
    main()
