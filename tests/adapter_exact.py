"""Inputs of the adapters whose outputs in 32 bits are known to the last bit, whatever the order of the sums (numpy).

``whole``: x, a, b and base are small integers and the scales powers of two.  Inner values are integers (halves) of up to 16
bits, which two bf16 terms hold (three: quarters at the least, eighths), and what is added to one output stays below 2^21: every
sum is exact, also where addends are cut off below 24 bits of the largest.  Each value that is left out, counted twice or
taken from another place shows, and a sum of zero is zero.

``single``: b has one power of two for each column, in another rank from column to column, and scales are of
all 24 bits: column j is the inner value j % rank, rounded to 32 bits once by its scale, times that power.  Three bf16 terms hold
it exactly (8 bits each), two to 2^-16.
"""
from __future__ import annotations

import numpy as np

BITS = {"bf16": 2.0 ** -16 + 2.0 ** -8 * (1 + 2.0 ** -16), "f32": 0.0}  # of ``single``: terms, then the output's rounding


def whole(tokens, count, k, n, rank, seed):
    assert 4 * k <= 2 ** 15  # inner values
    rng = np.random.default_rng(seed)
    x, a, b = (rng.integers(-2, 3, s).astype(np.int8) for s in ((tokens, k), (count, rank, k), (count, n, rank)))
    scale = 2.0 ** rng.integers(-1, 2, count)
    return x, a, b, scale.astype(np.float32), rng.integers(-9, 10, (tokens, n)).astype(np.int8), groups(tokens, count, rng)


def single(tokens, count, k, n, rank, seed):
    x, a, _, _, _, index = whole(tokens, count, k, 1, rank, seed)
    rng = np.random.default_rng(seed + 1)
    b = np.zeros((count, n, rank))
    for j in range(n):
        b[:, j, j % rank] = 2.0 ** rng.integers(-3, 4, count)
    return x, a, b, (rng.random(count) + 0.5).astype(np.float32), index


def groups(tokens, count, rng):
    """Adapters in runs of many lengths, a sixth of them without one; the first token has the last adapter."""
    index = np.empty(tokens, np.int32)
    at = 0
    while at < tokens:
        run = int(rng.integers(1, 2 + rng.choice([1, 6, 40, 300])))
        index[at:at + run] = rng.integers(count) if rng.random() < 5 / 6 else -1
        at += run
    index[0] = count - 1
    return index


def bf16(v):
    """Nearest bf16 values of 32-bit ones, ties to even, and those towards zero."""
    bits = np.asarray(v, np.float32).view(np.uint32)
    near = (bits + 0x7fff + (bits >> 16 & 1)) & np.uint32(0xffff0000)
    return near.view(np.float32), (bits & np.uint32(0xffff0000)).view(np.float32)


def terms(v, count):
    """The bf16 terms of 32-bit values as the kernels make them: cut off, in half where nothing would be left, the last rounded."""
    left, out = np.asarray(v, np.float32), []
    for _ in range(count - 1):
        cut = bf16(left)[1]
        half = np.float32(0.5) * left
        out.append(np.where(cut == left, half, cut))
        left = np.where(cut == left, half, left - np.where(cut == left, 0, cut))
    return out + [bf16(left)[0]]
