"""The operators of a linear layer trained and served in 8-bit floating point, as measured cases.

Four operators, each as a user's program calls it:

  quant    values to 8-bit floating point with a scale for each block of 128 (1 x 128 along a row, or
           128 x 128), row by row and, for training, transposed as well
  gemm     the product of two such operands, out[m][n] = sum_k a[m][k] b[n][k] with their scales
  ln_fwd   layer norm's forward pass: the rows, their means and reciprocal deviations
  ln_bwd   its backward pass: the input's gradient and, summed down the rows, the weight's and bias's

With ``own`` false ``run`` computes them in elementary torch operations in 32 bits; with ``own`` true
it calls ``shared_memory_tiled_gb300.binding``.
"""
import math

import torch

own = False

BLOCK = 128
FLOOR = 2.0 ** -100  # the least block maximum that a scale is made from
EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
TOP = {"e4m3": 448.0, "e5m2": 57344.0}  # the largest finite values


def listed():
    return [
        # one token's activations before a product
        {"name": "quant_token", "op": "quant", "rows": 1, "cols": 8192, "x": "bf16", "fp8": "e4m3", "block": 1, "both": False},
        # a training batch's activations: rows for the forward product, columns for the weight's gradient
        {"name": "quant_batch", "op": "quant", "rows": 16384, "cols": 8192, "x": "bf16", "fp8": "e4m3", "block": 1, "both": True},
        # a 32-bit master weight after an optimizer step, of odd sizes, for the forward and the backward product
        {"name": "quant_weight", "op": "quant", "rows": 12289, "cols": 7919, "x": "f32", "fp8": "e4m3", "block": 128, "both": True},
        # one token against a weight: bound by the weight's bytes
        {"name": "gemm_token", "op": "gemm", "m": 1, "n": 8192, "k": 8192, "a_block": 1, "b_block": 128, "a": "e4m3", "b": "e4m3", "out": "bf16"},
        # odd sizes everywhere: a ragged batch, a vocabulary-like width, a contraction that ends inside a block
        {"name": "gemm_odd", "op": "gemm", "m": 777, "n": 2049, "k": 1111, "a_block": 1, "b_block": 128, "a": "e4m3", "b": "e4m3", "out": "bf16"},
        # a training batch against a weight
        {"name": "gemm_batch", "op": "gemm", "m": 8192, "n": 8192, "k": 8192, "a_block": 1, "b_block": 128, "a": "e4m3", "b": "e4m3", "out": "bf16"},
        # a weight's gradient: both operands scaled along the tokens, the output in 32 bits
        {"name": "gemm_wgrad", "op": "gemm", "m": 4096, "n": 2048, "k": 16384, "a_block": 1, "b_block": 1, "a": "e5m2", "b": "e4m3", "out": "f32"},
        # one token's hidden state
        {"name": "ln_fwd_token", "op": "ln_fwd", "rows": 1, "cols": 8192, "x": "bf16", "w": "bf16", "bias": True},
        # a training batch
        {"name": "ln_fwd_batch", "op": "ln_fwd", "rows": 16384, "cols": 8192, "x": "bf16", "w": "f32", "bias": True},
        # a small model's micro batch
        {"name": "ln_bwd_small", "op": "ln_bwd", "rows": 256, "cols": 1024, "x": "bf16", "w": "f32", "bias": True},
        # 32-bit values, odd sizes, rows that start off 16-byte boundaries
        {"name": "ln_bwd_odd", "op": "ln_bwd", "rows": 12289, "cols": 7919, "x": "f32", "w": "f32", "bias": True},
        # a training batch
        {"name": "ln_bwd_batch", "op": "ln_bwd", "rows": 16384, "cols": 8192, "x": "bf16", "w": "f32", "bias": True},
    ]


def _size(rng, least, most):
    """A whole number between the two, spread over its logarithm; two in five are multiples of 128."""
    n = int(round(math.exp(rng.uniform(math.log(least), math.log(most)))))
    if rng.random() < 0.4 and n > BLOCK:
        n = n // BLOCK * BLOCK
    return max(least, min(most, n))


def draw(rng):
    op = rng.choice(["quant", "gemm", "gemm", "ln_fwd", "ln_bwd"])
    if op == "gemm":
        m, n, k = _size(rng, 1, 8192), _size(rng, 64, 8192), _size(rng, 128, 16384)
        while m * n * k > 8192 ** 3:
            k = max(128, k // 2)
        a_block, b_block = rng.choice([(1, 128), (1, 128), (1, 1), (128, 128)])
        return {"op": op, "m": m, "n": n, "k": k, "a_block": a_block, "b_block": b_block, "a": rng.choice(["e4m3", "e4m3", "e5m2"]),
                "b": "e4m3", "out": rng.choice(["bf16", "bf16", "f32"])}
    cols = _size(rng, 128, 16384)
    rows = _size(rng, 1, min(65536, 16384 * 8192 // cols))
    x = rng.choice(["bf16", "bf16", "f32"])
    if x == "f32":
        rows = max(1, rows // 2)
    if op == "quant":
        return {"op": op, "rows": rows, "cols": cols, "x": x, "fp8": rng.choice(["e4m3", "e4m3", "e5m2"]), "block": rng.choice([1, 1, 128]),
                "both": rng.random() < 0.6}
    return {"op": op, "rows": rows, "cols": cols, "x": x, "w": rng.choice(["f32", x]), "bias": rng.random() < 0.7}


def _up(n, to):
    return -(-n // to) * to


def _activations(rows, cols, gen):
    """Hidden states: a spread and an offset of its own for each channel, and a few channels that are far larger than the others."""
    spread = torch.exp(0.5 * torch.randn(cols, generator=gen, device="cuda"))
    spread = torch.where(torch.rand(cols, generator=gen, device="cuda") < 0.002, spread * 30, spread)
    offset = 0.3 + 0.2 * torch.randn(cols, generator=gen, device="cuda")
    return torch.randn(rows, cols, generator=gen, device="cuda").mul_(spread).add_(offset)


def _gradients(rows, cols, gen):
    """Gradients of hidden states: small, and of another size for each row."""
    size = 1e-3 * torch.exp(torch.randn(rows, 1, generator=gen, device="cuda"))
    return torch.randn(rows, cols, generator=gen, device="cuda").mul_(size)


def _blocks(x, block):
    """x[rows][cols] padded with zeros to whole blocks, as [row blocks][block rows][column blocks][128]."""
    rows, cols = x.shape
    up = torch.zeros(_up(rows, block), _up(cols, BLOCK), dtype=torch.float32, device=x.device)
    up[:rows, :cols] = x
    return up.view(up.shape[0] // block, block, up.shape[1] // BLOCK, BLOCK)


def _plain_quant(x, fp8, block):
    """(values in 8 bits, scales [column blocks][row blocks])"""
    rows, cols = x.shape
    up = _blocks(x, block)
    most = up.abs().amax(dim=(1, 3)).clamp(min=FLOOR)
    scale, inverse = most / TOP[fp8], TOP[fp8] / most
    q = (up * inverse[:, None, :, None]).view(-1, up.shape[2] * BLOCK)[:rows, :cols].to(FP8[fp8])
    return q, scale.t().contiguous()


def _plain_values(q, scale):
    """What 8-bit values with their scales stand for, in 32 bits."""
    rows, cols = q.shape
    block = 1 if scale.shape[1] == rows else BLOCK
    return q.to(torch.float32) * scale.t().repeat_interleave(block, 0)[:rows].repeat_interleave(BLOCK, 1)[:, :cols]


def _operand(rows, cols, fp8, block, gen):
    """An operand of a product as quantizing leaves it: its rows start on 16-byte boundaries."""
    x = _gradients(rows, cols, gen) if fp8 == "e5m2" else 0.02 * torch.randn(rows, cols, generator=gen, device="cuda") if block == 128 else _activations(rows, cols, gen)
    q, scale = _plain_quant(x, fp8, block)
    held = torch.zeros(rows, _up(cols, 16), dtype=torch.uint8, device="cuda").view(FP8[fp8])[:, :cols]
    held.view(torch.uint8).copy_(q.view(torch.uint8))
    return held, scale


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case)
    if case["op"] == "gemm":
        s["qa"], s["sa"] = _operand(case["m"], case["k"], case["a"], case["a_block"], gen)
        s["qb"], s["sb"] = _operand(case["n"], case["k"], case["b"], case["b_block"], gen)
        return s
    rows, cols = case["rows"], case["cols"]
    x = 0.02 * torch.randn(rows, cols, generator=gen, device="cuda") if case.get("block") == 128 else _activations(rows, cols, gen)
    if case["op"] == "quant":
        if case["fp8"] == "e5m2" and case["block"] == 1:
            x = _gradients(rows, cols, gen)
        s["x"] = x.to(TYPES[case["x"]])
        return s
    s["x"] = x.to(TYPES[case["x"]])
    s["gamma"] = (1 + 0.1 * torch.randn(cols, generator=gen, device="cuda")).to(TYPES[case["w"]])
    s["beta"] = (0.1 * torch.randn(cols, generator=gen, device="cuda")).to(TYPES[case["w"]]) if case["bias"] else None
    if case["op"] == "ln_bwd":
        s["dy"] = _gradients(rows, cols, gen).to(TYPES[case["x"]])
        x = s["x"].to(torch.float32)
        s["mean"] = x.mean(1)
        s["rstd"] = (x - s["mean"][:, None]).square_().mean(1).add_(EPS).rsqrt_()
    return s


def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    from shared_memory_tiled_gb300 import binding as B
    op = s["op"]
    if op == "quant":
        return B.quantize_fp8(s["x"], dtype=FP8[s["fp8"]], block_rows=s["block"], transposed=s["both"])
    if op == "gemm":
        return B.matmul_fp8(s["qa"], s["sa"], s["qb"], s["sb"], out_dtype=TYPES[s["out"]])
    if op == "ln_fwd":
        return B.layernorm(s["x"], s["gamma"], s["beta"], eps=EPS)
    return B.layernorm_backward(s["dy"], s["x"], s["gamma"], s["mean"], s["rstd"], bias=s["bias"])


def _run_plain(s):
    op = s["op"]
    if op == "quant":
        got = _plain_quant(s["x"], s["fp8"], s["block"])
        return got + _plain_quant(s["x"].t(), s["fp8"], s["block"]) if s["both"] else got
    if op == "gemm":
        return torch.matmul(_plain_values(s["qa"], s["sa"]), _plain_values(s["qb"], s["sb"]).t()).to(TYPES[s["out"]])
    x, gamma = s["x"].to(torch.float32), s["gamma"].to(torch.float32)
    if op == "ln_fwd":
        mean = x.mean(1)
        off = x - mean[:, None]
        rstd = 1 / torch.sqrt((off * off).mean(1) + EPS)
        y = off * rstd[:, None] * gamma
        if s["beta"] is not None:
            y = y + s["beta"].to(torch.float32)
        return y.to(s["x"].dtype), mean, rstd
    dy = s["dy"].to(torch.float32)
    unit = (x - s["mean"][:, None]) * s["rstd"][:, None]
    g = dy * gamma
    dx = s["rstd"][:, None] * (g - g.mean(1, keepdim=True) - unit * (g * unit).mean(1, keepdim=True))
    return dx.to(s["x"].dtype), (dy * unit).sum(0), dy.sum(0) if s["bias"] else None


def work(case):
    if case["op"] == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        kb = -(-k // BLOCK)
        scales = 4 * kb * (-(-m // case["a_block"]) + -(-n // case["b_block"]))
        return {"bytes": m * k + n * k + scales + m * n * (2 if case["out"] == "bf16" else 4), "flops": 2 * m * n * k}
    rows, cols, size = case["rows"], case["cols"], 2 if case["x"] == "bf16" else 4
    if case["op"] == "quant":
        b = case["block"]
        scales = 4 * (-(-cols // BLOCK) * -(-rows // b) + (-(-rows // BLOCK) * -(-cols // b) if case["both"] else 0))
        outs = 2 if case["both"] else 1
        return {"bytes": rows * cols * (size + outs) + scales, "flops": rows * cols * (1 + outs if b == 128 else 2 * outs)}
    w = 2 if case["w"] == "bf16" else 4
    if case["op"] == "ln_fwd":
        return {"bytes": 2 * rows * cols * size + cols * w * (2 if case["bias"] else 1) + 8 * rows, "flops": 8 * rows * cols}
    return {"bytes": 3 * rows * cols * size + cols * (w + 4 * (2 if case["bias"] else 1)) + 8 * rows, "flops": 14 * rows * cols}


def _exact_quant(x, fp8, block):
    """The same from the definition in 64 bits; the rounding to 8 bits is written out, to the nearest of its values and ties to even."""
    rows, cols = x.shape
    kept, least = (3, -6) if fp8 == "e4m3" else (2, -14)  # bits of the fraction, exponent of the smallest normal value
    rb, cb = -(-rows // block), -(-cols // BLOCK)
    up = torch.nn.functional.pad(x.double(), (0, cb * BLOCK - cols, 0, rb * block - rows)).reshape(rb, block, cb, BLOCK)
    scale = torch.clamp(up.abs().amax(3).amax(1), min=FLOOR) / TOP[fp8]
    v = up / scale[:, None, :, None]
    exponent = torch.clamp(torch.frexp(v)[1] - 1, min=least).double()
    step = torch.exp2(exponent - kept)
    v = torch.clamp(torch.round(v / step) * step, -TOP[fp8], TOP[fp8])
    return v.reshape(rb * block, cb * BLOCK)[:rows, :cols], scale.t().contiguous()


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quant":
        got = _exact_quant(s["x"], s["fp8"], s["block"])
        return got + _exact_quant(s["x"].t(), s["fp8"], s["block"]) if s["both"] else got
    if case["op"] == "gemm":
        def values(q, scale, block):
            rows, cols = q.shape
            at = torch.arange(rows, device="cuda") // block, torch.arange(cols, device="cuda") // BLOCK
            return q.double() * scale.double()[at[1][None, :], at[0][:, None]]
        return values(s["qa"], s["sa"], case["a_block"]) @ values(s["qb"], s["sb"], case["b_block"]).t()
    x, gamma = s["x"].double(), s["gamma"].double()
    if case["op"] == "ln_fwd":
        variance, mean = torch.var_mean(x, 1, correction=0)
        rstd = (variance + EPS) ** -0.5
        y = (x - mean[:, None]) * rstd[:, None] * gamma
        return y if s["beta"] is None else y + s["beta"].double(), mean, rstd
    n, dy, rstd = case["cols"], s["dy"].double(), s["rstd"].double()[:, None]
    unit = (x - s["mean"].double()[:, None]) * rstd
    g = dy * gamma
    dx = rstd / n * (n * g - g.sum(1)[:, None] - unit * (g * unit).sum(1)[:, None])
    return dx, (dy * unit).sum(0), dy.sum(0) if s["bias"] else None
