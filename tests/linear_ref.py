"""Plain 64-bit forms of the linear layer's operators, and how far a 32-bit
result may be from them.

Everything here is numpy (or torch on the CPU) written from the definitions in
``include/transpose.h``; nothing of the library is used.  Bounds: a sum of n
terms in 32 bits, in any order, is within (depth) * 2^-24 * sum |terms| of the
exact one, with depth the longest chain of additions; each further operation
adds 2^-24 of its result, and an output held in bf16 2^-8 of itself.
"""
from __future__ import annotations

import numpy as np

U32 = 2.0 ** -24   # unit roundoff, 32 bits
U16 = 2.0 ** -8    # unit roundoff, bf16 (8 significant bits)
FLOOR = np.float32(2.0 ** -100)
TOP = {"e4m3": np.float32(448.0), "e5m2": np.float32(57344.0)}


def fp8(x32: np.ndarray, kind: str) -> np.ndarray:
    """32-bit values to 8 bits (as uint8), nearest with ties to even, magnitudes
    limited to the largest finite value; the rounding is written out on integers
    of 1/8 (e5m2: 1/4) of a binade."""
    keep, least = (3, -6) if kind == "e4m3" else (2, -14)
    x = x32.astype(np.float64)
    sign = np.signbit(x).astype(np.uint8) << 7
    a = np.minimum(np.abs(x), float(TOP[kind]))
    nan = np.isnan(x)
    a = np.where(nan, 0.0, a)
    e = np.where(a > 0, np.maximum(np.frexp(a)[1] - 1, least), least)
    n = np.rint(np.ldexp(a, keep - e))            # ties to even
    code = (e - least) * (1 << keep) + n          # a carry moves into the exponent by itself
    code = np.minimum(code, 0x7E if kind == "e4m3" else 0x7B).astype(np.uint8)
    return np.where(nan, np.uint8(0x7F), sign | code)


def fp8_values(q: np.ndarray, kind: str) -> np.ndarray:
    """8-bit codes as 64-bit values."""
    keep, least = (3, -6) if kind == "e4m3" else (2, -14)
    code = (q & 0x7F).astype(np.int64)
    e, m = code >> keep, code & ((1 << keep) - 1)
    v = np.where(e == 0, np.ldexp(m.astype(float), least - keep),
                 np.ldexp((m + (1 << keep)).astype(float), np.maximum(e, 1) - 1 + least - keep))
    if kind == "e4m3":
        v = np.where(code == 0x7F, np.nan, v)
    else:
        v = np.where(code == 0x7C, np.inf, np.where(code > 0x7C, np.nan, v))
    return np.where(q & 0x80, -v, v)


def quantize(x: np.ndarray, kind: str, block: int):
    """(codes, scales [column blocks][row blocks]) by the header's 32-bit formula."""
    rows, cols = x.shape
    rb, cb = -(-rows // block), -(-cols // 128)
    up = np.zeros((rb * block, cb * 128), np.float32)
    up[:rows, :cols] = x
    up = up.reshape(rb, block, cb, 128)
    with np.errstate(all="ignore"):
        most = np.abs(up).max(axis=(1, 3))           # NaN wins
        a = np.where(np.isnan(most), most, np.maximum(most, FLOOR)).astype(np.float32)
        scale, inverse = a / TOP[kind], TOP[kind] / a
        q = fp8(up * inverse[:, None, :, None], kind)
    return q.reshape(rb * block, cb * 128)[:rows, :cols], np.ascontiguousarray(scale.T)


def dequantize(q: np.ndarray, scale: np.ndarray, kind: str, block: int) -> np.ndarray:
    rows, cols = q.shape
    s = scale.astype(np.float64).T.repeat(block, 0)[:rows].repeat(128, 1)[:, :cols]
    return fp8_values(q, kind) * s


def matmul(a, sa, ka, ab, b, sb, kb, bb):
    """(exact product, bound on a 32-bit result's error).  A block's 128 products
    are summed by the tensor cores, whose additions may truncate (one unit in
    the last place, 2^-23, each); blocks follow one another, at most 8 parts
    are joined."""
    x, y = dequantize(a, sa, ka, ab), dequantize(b, sb, kb, bb)
    blocks = -(-x.shape[1] // 128)
    return x @ y.T, (128 * 2 + blocks + 8 + 4) * U32 * (np.abs(x) @ np.abs(y).T)


def layernorm(x, gamma, beta, eps):
    """(y, mean, rstd, bounds on each) in 64 bits."""
    x = x.astype(np.float64)
    cols = x.shape[1]
    mean = x.mean(1, keepdims=True)
    rstd = 1 / np.sqrt(((x - mean) ** 2).mean(1, keepdims=True) + eps)
    u = (x - mean) * rstd
    y = u * gamma + (0 if beta is None else beta)
    depth = 64 + cols / 256                       # a thread's own values, then 10 levels of a tree
    dm = depth * U32 * np.abs(x).mean(1, keepdims=True) + U32 * np.abs(mean)
    # variance: the sum's own error, and each deviation's by the mean's error and one rounding
    dev = np.abs(x - mean)
    dv = (depth + 4) * U32 * (dev ** 2).mean(1, keepdims=True) + 2 * dev.mean(1, keepdims=True) * dm + dm ** 2
    dr = rstd * (0.5 * dv * rstd ** 2 + 4 * U32)
    dy = np.abs(gamma) * (rstd * (dm + U32 * dev) + dev * dr + 4 * U32 * np.abs(u)) + 2 * U32 * np.abs(y)
    return y, mean[:, 0], rstd[:, 0], dy, dm[:, 0], dr[:, 0]


def layernorm_backward(dy, x, gamma, mean, rstd):
    """(dx, dgamma, dbeta, bounds on each) in 64 bits from the given statistics."""
    dy, x = dy.astype(np.float64), x.astype(np.float64)
    rows, cols = x.shape
    mean, rstd = mean.astype(np.float64)[:, None], rstd.astype(np.float64)[:, None]
    u = (x - mean) * rstd
    g = dy * gamma
    c1, c2 = g.mean(1, keepdims=True), (g * u).mean(1, keepdims=True)
    dx = rstd * (g - c1 - u * c2)
    depth = 64 + cols / 256
    du = 2 * U32 * np.abs(u)
    e1 = (depth + 2) * U32 * np.abs(g).mean(1, keepdims=True)
    e2 = (depth + 6) * U32 * np.abs(g * u).mean(1, keepdims=True)
    ex = rstd * (4 * U32 * (np.abs(g) + np.abs(c1) + np.abs(u * c2)) + e1 + np.abs(u) * e2 + du * np.abs(c2))
    # down a column: at most every row in one chain
    return (dx, (dy * u).sum(0), dy.sum(0), ex, (rows + 8) * U32 * np.abs(dy * u).sum(0),
            (rows + 2) * U32 * np.abs(dy).sum(0))
