"""Plain 64-bit forms of root-mean-square norm, its backward pass and the adapters, and how far a
32-bit result may be from them (numpy, from the definitions in ``include/transpose.h``).

Bounds are derived as in ``linear_ref``: a sum of n terms in 32 bits is within (longest chain of
additions) * 2^-24 * sum |terms|, each further operation adds 2^-24 of its result.
"""
from __future__ import annotations

import numpy as np

import linear_ref as R

U32 = R.U32


def rmsnorm(h, gamma, eps):
    """(y, rstd, bounds on each before y is rounded) in 64 bits."""
    h = h.astype(np.float64)
    cols = h.shape[1]
    rstd = 1 / np.sqrt((h ** 2).mean(1, keepdims=True) + eps)
    y = h * rstd * gamma
    depth = 64 + cols / 256                  # a thread's own values, then 10 levels of a tree
    # the sum with its squares' roundings, 1/n and the product with it, the addition of eps: all
    # positive, so relative; the root halves that; root, quotient
    rel = 0.5 * (depth + 4) * U32 + 2 * U32
    return y, rstd[:, 0], np.abs(y) * (rel + 3 * U32), rstd[:, 0] * rel


def check_quantized(codes, scale, y, dy, kind):
    """8-bit codes [rows][cols] and scales [blocks][rows] of y (64 bits, known to +-dy before it is
    quantized in 32 bits): each scale within its bound, each code the right one where the
    uncertainty does not reach over a border between two codes, else one of the two."""
    rows, cols = y.shape
    blocks = -(-cols // 128)
    up = np.zeros((rows, blocks * 128))
    up[:, :cols] = np.abs(y)
    top = float(R.TOP[kind])
    rel = float(np.max(dy / np.maximum(np.abs(y), 1e-300))) if y.size else 0.0
    amax = np.maximum(up.reshape(rows, blocks, 128).max(2), float(R.FLOOR))
    want = (amax / top).T
    assert np.all(np.abs(scale - want) <= want * (rel + 2 * U32)), "scales"
    t = y / (amax / top).repeat(128, 1)[:, :cols]
    slack = 2 * rel + 4 * U32                # y's own, the maximum's, T / a and the product with it
    low, high = R.fp8(t * (1 - slack), kind), R.fp8(t * (1 + slack), kind)
    ok = (codes == low) | (codes == high)
    assert ok.all(), (f"{(~ok).sum()} codes of {ok.size}, first at {np.argwhere(~ok)[0]}")


def rmsnorm_backward(dy, h, gamma, rstd, dres):
    """(dx, dgamma, bounds on each) in 64 bits from the given rstd."""
    dy, h = dy.astype(np.float64), h.astype(np.float64)
    rows, cols = h.shape
    rstd = rstd.astype(np.float64)[:, None]
    u, g = h * rstd, dy * gamma
    c = (g * u).mean(1, keepdims=True)
    dx = rstd * (g - u * c) + (0 if dres is None else dres)
    depth = 64 + cols / 256
    ec = (depth + 6) * U32 * np.abs(g * u).mean(1, keepdims=True)
    ex = rstd * (5 * U32 * (np.abs(g) + np.abs(u * c)) + np.abs(u) * ec) + 2 * U32 * np.abs(dx)
    return dx, (dy * u).sum(0), ex, (rows + 8) * U32 * np.abs(dy * u).sum(0)


def adapters(x, a, b, scale, index, base):
    """(out, bound before out is rounded) in 64 bits.  The inner values' sums may truncate (2^-23 each),
    they are held in 16 bits (2^-16), and the outer sums have three terms at most to each of them."""
    x, a, b = (v.astype(np.float64) for v in (x, a, b))
    tokens, k = x.shape
    count, n, rank = b.shape
    out = np.zeros((tokens, n)) if base is None else base.astype(np.float64).copy()
    bound = np.zeros((tokens, n))
    for g in range(count):
        at = np.flatnonzero(index == g)
        if not at.size:
            continue
        v, size = scale[g] * (x[at] @ a[g].T), abs(scale[g]) * (np.abs(x[at]) @ np.abs(a[g]).T)
        dv = (2 * k + 8) * U32 * size + 2.0 ** -16 * np.abs(v)
        out[at] += v @ b[g].T
        bound[at] = dv @ np.abs(b[g]).T + (6 * rank + 2) * U32 * (np.abs(v) @ np.abs(b[g]).T) + U32 * np.abs(out[at])
    return out, bound
