"""The operators before and beside the 8-bit linear layer of a model, as measured cases.

Four operators, each as a user's program calls it:

  norm    root-mean-square norm of the residual stream with a branch added to it: the rows, the new
          stream and the rows' reciprocal root mean squares
  norm8   the same, with the rows in 8-bit floating point and a scale for each block of 128, as the
          product takes them; for training transposed as well
  back    the norm's backward pass: the gradient of the stream (what already flows into it added) and,
          summed down the rows, the weight's
  adapt   low-rank adapters of many requests beside a shared projection: out = base + s_g B_g A_g x
          for each token x and the adapter g of its request, with the grouping of the tokens

With ``own`` false ``run`` computes them in elementary torch operations in 32 bits; with ``own`` true
it calls ``shared_memory_tiled_gb300.binding``.
"""
import math

import torch

own = False

BLOCK = 128
FLOOR = 2.0 ** -100  # the least block maximum that a scale is made from
TOP = 448.0          # the largest value of 8-bit floating point with 4 bits of exponent
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one token's hidden state between two layers
        {"name": "norm_token", "op": "norm", "rows": 1, "cols": 8192, "x": "bf16", "w": "bf16", "add": True},
        # 32-bit values, odd sizes, rows that start off 16-byte boundaries
        {"name": "norm_odd", "op": "norm", "rows": 12289, "cols": 7919, "x": "f32", "w": "f32", "add": True},
        # a training batch between two layers
        {"name": "norm_batch", "op": "norm", "rows": 16384, "cols": 8192, "x": "bf16", "w": "f32", "add": True},
        # one token before an 8-bit product
        {"name": "norm8_token", "op": "norm8", "rows": 1, "cols": 8192, "x": "bf16", "w": "bf16", "add": True, "both": False},
        # a training batch before an 8-bit product: rows for the forward pass, columns for the weight's gradient
        {"name": "norm8_batch", "op": "norm8", "rows": 16384, "cols": 8192, "x": "bf16", "w": "f32", "add": True, "both": True},
        # a small model's micro batch, its first layer: nothing else flows into the stream
        {"name": "back_small", "op": "back", "rows": 256, "cols": 1024, "x": "bf16", "w": "f32", "add": False},
        # 32-bit values, odd sizes, rows that start off 16-byte boundaries
        {"name": "back_odd", "op": "back", "rows": 12289, "cols": 7919, "x": "f32", "w": "f32", "add": True},
        # a training batch
        {"name": "back_batch", "op": "back", "rows": 16384, "cols": 8192, "x": "bf16", "w": "f32", "add": True},
        # one request's next token
        {"name": "adapt_token", "op": "adapt", "requests": 1, "tokens": 1, "bare": 0, "k": 8192, "n": 8192, "rank": 16, "adapters": 32, "outs": 1, "out": "bf16"},
        # the next tokens of 64 requests, most with an adapter of their own, into the three projections before attention
        {"name": "adapt_decode", "op": "adapt", "requests": 64, "tokens": 64, "bare": 5, "k": 8192, "n": 8192, "rank": 16, "adapters": 48, "outs": 3, "out": "bf16"},
        # odd sizes everywhere: ragged prompts, one without an adapter, a rank that fills no tile, a 32-bit output
        {"name": "adapt_odd", "op": "adapt", "requests": 7, "tokens": 777, "bare": 1, "k": 1111, "n": 2049, "rank": 12, "adapters": 5, "outs": 1, "out": "f32"},
        # a batch of long prompts
        {"name": "adapt_prompts", "op": "adapt", "requests": 9, "tokens": 8192, "bare": 1, "k": 8192, "n": 8192, "rank": 64, "adapters": 8, "outs": 1, "out": "bf16"},
    ]


def _size(rng, least, most):
    """A whole number between the two, spread over its logarithm; two in five are multiples of 128."""
    n = int(round(math.exp(rng.uniform(math.log(least), math.log(most)))))
    if rng.random() < 0.4 and n > BLOCK:
        n = n // BLOCK * BLOCK
    return max(least, min(most, n))


def draw(rng):
    op = rng.choice(["norm", "norm8", "back", "adapt", "adapt"])
    if op == "adapt":
        tokens, rank, adapters = _size(rng, 1, 8192), _size(rng, 4, 128), _size(rng, 1, 64)
        k, n = _size(rng, 128, 8192), _size(rng, 64, 8192)
        while max(tokens, 512) * (k + n) * rank * adapters > 8192 * 16384 * 512:
            adapters, rank = max(1, adapters // 2), max(4, rank * 3 // 4)
        # next tokens of as many requests, or a few prompts
        requests = tokens if tokens <= 256 and rng.random() < 0.7 else rng.randint(1, min(tokens, 16))
        return {"op": op, "requests": requests, "tokens": tokens, "bare": min(requests - 1, rng.choice([0, 0, 1, 3])), "k": k, "n": n, "rank": rank,
                "adapters": adapters, "outs": rng.choice([1, 1, 3]) if tokens <= 256 else 1, "out": rng.choice(["bf16", "bf16", "f32"])}
    cols = _size(rng, 128, 16384)
    rows = _size(rng, 1, min(65536, 16384 * 8192 // cols))
    x = rng.choice(["bf16", "bf16", "f32"])
    if x == "f32":
        rows = max(1, rows // 2)
    case = {"op": op, "rows": rows, "cols": cols, "x": x, "w": rng.choice(["f32", x]), "add": rng.random() < 0.7}
    if op == "norm8":
        case["both"] = rng.random() < 0.5
    return case


def _activations(rows, cols, gen):
    """Hidden states: a spread of its own for each channel, and a few channels that are far larger than the others."""
    spread = torch.exp(0.5 * torch.randn(cols, generator=gen, device="cuda"))
    spread = torch.where(torch.rand(cols, generator=gen, device="cuda") < 0.002, spread * 30, spread)
    return torch.randn(rows, cols, generator=gen, device="cuda").mul_(spread)


def _gradients(rows, cols, gen):
    """Gradients of hidden states: small, and of another size for each row."""
    size = 1e-3 * torch.exp(torch.randn(rows, 1, generator=gen, device="cuda"))
    return torch.randn(rows, cols, generator=gen, device="cuda").mul_(size)


def _held(values):
    """The same in bf16, rows on 16-byte boundaries, as a program holds what a product reads."""
    cols = values.shape[-1]
    held = torch.zeros(*values.shape[:-1], -(-cols // 8) * 8, dtype=torch.bfloat16, device="cuda")
    held[..., :cols] = values
    return held[..., :cols]


def _used(case):
    """Adapters that some request has."""
    return min(case["adapters"], case["requests"] - case["bare"])


def _prepare_adapt(s, case, gen):
    requests, tokens, adapters = case["requests"], case["tokens"], case["adapters"]
    # Which adapter each request has (-1: none), in no order; how many tokens each brings.
    of = torch.arange(requests, device="cuda") % adapters
    of[requests - case["bare"]:] = -1
    of = of[torch.randperm(requests, generator=gen, device="cuda")]
    share = torch.rand(requests, generator=gen, device="cuda") + 0.1
    ends = torch.arange(1, requests + 1, device="cuda") + (share.cumsum(0) / share.sum() * (tokens - requests) + 1e-3).long().clamp(max=tokens - requests)
    ends[-1] = tokens
    s["index"] = of[torch.searchsorted(ends, torch.arange(tokens, device="cuda"), right=True)].to(torch.int32)
    k, n, rank = case["k"], case["n"], case["rank"]
    s["x"] = _held(_activations(tokens, k, gen))
    s["scale"] = torch.rand(adapters, generator=gen, device="cuda") + 0.5
    s["sets"] = []
    for _ in range(case["outs"]):
        a = _held(torch.randn(adapters, rank, k, generator=gen, device="cuda") / k ** 0.5)
        b = _held(0.1 * torch.randn(adapters, n, rank, generator=gen, device="cuda") / rank ** 0.5)
        base = torch.randn(tokens, n, generator=gen, device="cuda").to(TYPES[case["out"]])
        s["sets"].append((a, b, base))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case)
    if case["op"] == "adapt":
        _prepare_adapt(s, case, gen)
        return s
    rows, cols, kind = case["rows"], case["cols"], TYPES[case["x"]]
    s["gamma"] = (1 + 0.1 * torch.randn(cols, generator=gen, device="cuda")).to(TYPES[case["w"]])
    x = _activations(rows, cols, gen).to(kind)
    if case["op"] == "back":
        s["h"] = x
        s["rstd"] = (x.to(torch.float32).square().mean(1) + EPS).rsqrt_()
        s["dy"] = _gradients(rows, cols, gen).to(kind)
        s["dh"] = _gradients(rows, cols, gen).to(kind) if case["add"] else None
        return s
    s["x"] = x
    s["residual"] = (4 * _activations(rows, cols, gen)).to(kind) if case["add"] else None
    return s


def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    from shared_memory_tiled_gb300 import binding as B
    op = s["op"]
    if op == "norm":
        return B.rmsnorm(s["x"], s["gamma"], s["residual"], eps=EPS)
    if op == "norm8":
        return B.rmsnorm_fp8(s["x"], s["gamma"], s["residual"], eps=EPS, transposed=s["both"])
    if op == "back":
        return B.rmsnorm_backward(s["dy"], s["h"], s["gamma"], s["rstd"], dresidual=s["dh"])
    plan = B.adapter_plan(s["index"], s["adapters"])
    return [B.adapters(s["x"], a, b, plan, scale=s["scale"], base=base) for a, b, base in s["sets"]]


def _plain_quant(x):
    """(values in 8 bits, scales [column blocks][rows]) for blocks of 128 along the rows."""
    rows, cols = x.shape
    up = torch.zeros(rows, -(-cols // BLOCK) * BLOCK, dtype=torch.float32, device=x.device)
    up[:, :cols] = x
    up = up.view(rows, -1, BLOCK)
    most = up.abs().amax(dim=2).clamp(min=FLOOR)
    q = (up * (TOP / most)[:, :, None]).view(rows, -1)[:, :cols].to(torch.float8_e4m3fn)
    return q, (most / TOP).t().contiguous()


def _run_plain(s):
    op = s["op"]
    if op == "adapt":
        return [_plain_adapt(s, a, b, base) for a, b, base in s["sets"]]
    gamma = s["gamma"].to(torch.float32)
    if op == "back":
        dy, rstd = s["dy"].to(torch.float32), s["rstd"][:, None]
        unit = s["h"].to(torch.float32) * rstd
        g = dy * gamma
        dx = rstd * (g - unit * (g * unit).mean(1, keepdim=True))
        if s["dh"] is not None:
            dx = dx + s["dh"].to(torch.float32)
        return dx.to(s["h"].dtype), (dy * unit).sum(0)
    h = s["x"]
    if s["residual"] is not None:
        h = (h.to(torch.float32) + s["residual"].to(torch.float32)).to(h.dtype)
    wide = h.to(torch.float32)
    rstd = 1 / torch.sqrt((wide * wide).mean(1) + EPS)
    y = wide * rstd[:, None] * gamma
    if op == "norm":
        return y.to(h.dtype), h, rstd
    return _plain_quant(y) + (_plain_quant(y.t()) if s["both"] else ()) + (h, rstd)


def _plain_adapt(s, a, b, base):
    """All adapters' inner values for all tokens, those of another adapter than the token's taken out."""
    adapters, rank, k = a.shape
    inner = torch.matmul(s["x"].to(torch.float32), a.to(torch.float32).reshape(adapters * rank, k).t())
    of = torch.arange(adapters, device=a.device).repeat_interleave(rank)
    inner = torch.where(s["index"][:, None] == of, inner * s["scale"].repeat_interleave(rank), 0.0)
    up = b.to(torch.float32).permute(0, 2, 1).reshape(adapters * rank, b.shape[1])
    return (base.to(torch.float32) + torch.matmul(inner, up)).to(base.dtype)


def work(case):
    if case["op"] == "adapt":
        t, k, n, r, outs, used = case["tokens"], case["k"], case["n"], case["rank"], case["outs"], _used(case)
        size = 2 if case["out"] == "bf16" else 4
        carried = t if not case["bare"] else t * (case["requests"] - case["bare"]) / case["requests"]  # tokens with an adapter, about
        return {"bytes": 2 * t * k + 4 * t + 4 * used + outs * (2 * used * r * (k + n) + 2 * size * t * n), "flops": outs * carried * 2 * r * (k + n)}
    rows, cols, size = case["rows"], case["cols"], 2 if case["x"] == "bf16" else 4
    w = 2 if case["w"] == "bf16" else 4
    if case["op"] == "back":
        return {"bytes": (4 if case["add"] else 3) * rows * cols * size + cols * (w + 4) + 4 * rows, "flops": 11 * rows * cols}
    through = rows * cols * size * (3 if case["add"] else 1) + cols * w + 4 * rows  # x, and with a residual that and the new stream
    if case["op"] == "norm":
        return {"bytes": through + rows * cols * size, "flops": 5 * rows * cols}
    scales = 4 * (-(-cols // BLOCK) * rows + (-(-rows // BLOCK) * cols if case["both"] else 0))
    outs = 2 if case["both"] else 1
    return {"bytes": through + outs * rows * cols + scales, "flops": (5 + 2 * outs) * rows * cols}


def _exact_quant(x):
    """The same from the definition; the rounding to 8 bits is written out, to the nearest of its values and ties to even."""
    rows, cols = x.shape
    up = torch.nn.functional.pad(x, (0, -cols % BLOCK)).unflatten(1, (-1, BLOCK))
    scale = torch.clamp(up.abs().amax(2), min=FLOOR) / TOP
    v = up / scale[:, :, None]
    step = torch.exp2(torch.clamp(torch.frexp(v)[1] - 1, min=-6).double() - 3)
    v = torch.clamp(torch.round(v / step) * step, -TOP, TOP)
    return v.flatten(1)[:, :cols], scale.t().contiguous()


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "adapt":
        got = []
        for a, b, base in s["sets"]:
            out = base.double()
            for g in torch.unique(s["index"]).tolist():
                if g >= 0:
                    at = torch.nonzero(s["index"] == g)[:, 0]
                    out[at] += float(s["scale"][g]) * (s["x"][at].double() @ a[g].double().t() @ b[g].double().t())
            got.append(out)
        return got
    gamma, n = s["gamma"].double(), case["cols"]
    if case["op"] == "back":
        dy, h, rstd = s["dy"].double(), s["h"].double(), s["rstd"].double()
        along = torch.einsum("ij,ij,j->i", dy, h, gamma)
        dx = dy * gamma * rstd[:, None] - h * (along * rstd ** 3 / n)[:, None]
        return dx if s["dh"] is None else dx + s["dh"].double(), torch.einsum("ij,ij,i->j", dy, h, rstd)
    h = s["x"]
    if s["residual"] is not None:
        h = torch.add(h.double(), s["residual"].double()).to(h.dtype)  # the stream is what its type holds
    norm = torch.linalg.vector_norm(h.double(), dim=1)
    rstd = (norm ** 2 / n + EPS) ** -0.5
    y = torch.einsum("ij,i,j->ij", h.double(), rstd, gamma)
    if case["op"] == "norm":
        return y, h.double(), rstd
    return _exact_quant(y) + (_exact_quant(y.t()) if case["both"] else ()) + (h.double(), rstd)
