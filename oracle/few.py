"""The expert block for a few tokens: W1, SwiGLU, W2 and the weighted sum, from dequantized weights.

TEST INFRASTRUCTURE ONLY (see the package docstring).

With [g | u] = x[t] W1[e]^T and a = bf16(silu(g) * u), y[t] = sum over the experts e that ids[t] names of
(the sum of the weights of those slots) * a W2[e]^T.  Everything but a's rounding is fp64; ``bounds`` says how far an fp32
evaluation that rounds a itself may be from it.
"""
from __future__ import annotations

import numpy as np

from .quant import bf16_to_f32
from .swiglu import round_bf16


def silu(g: np.ndarray) -> np.ndarray:
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g))


def block(x: np.ndarray, ids: np.ndarray, weights: np.ndarray, w1: np.ndarray, w2: np.ndarray):
    """x fp64 [T, K], ids [T, k], weights [T, k], w1 fp64 [E, 2F, K], w2 fp64 [E, K, F] -> (y [T, K], bound [T, K]).

    The bound: a sum of n fp32 products is within (n + 8) 2^-23 of the sum of their magnitudes (products of bf16 values
    are exact in fp32; a matrix instruction may truncate where an addition rounds, and the waves' sums and the
    scale's division are within the eight).  silu's slope is at most 1.1, its own evaluation and the product by u within
    2^-20.  Where that leaves a's rounding to bf16 open it may go the other way, one step of 2^-7 of its magnitude; elsewhere a
    is the reference's.  y's bf16 rounding comes on top."""
    T, K = x.shape
    E, F = w1.shape[0], w1.shape[1] // 2
    y, err = np.zeros((T, K)), np.zeros((T, K))
    for e in range(E):
        wt = np.where(ids == e, weights, 0.0).sum(axis=1)
        use = (ids == e).any(axis=1)
        if not use.any():
            continue
        h = x[use] @ w1[e].T
        dh = (K + 8) * 2.0 ** -23 * (np.abs(x[use]) @ np.abs(w1[e]).T)
        g, u, dg, du = h[:, :F], h[:, F:], dh[:, :F], dh[:, F:]
        s = silu(g)
        a = s * u
        da = 1.1 * dg * (np.abs(u) + du) + np.abs(s) * du + 2.0 ** -20 * np.abs(a) + 1e-38
        lo, hi = (bf16_to_f32(round_bf16(v)).astype(np.float64) for v in (a - da, a + da))
        ar = bf16_to_f32(round_bf16(a)).astype(np.float64)
        step = np.maximum(np.abs(hi - ar), np.abs(ar - lo))     # zero where both ends round alike
        o = ar @ w2[e].T
        do = step @ np.abs(w2[e]).T + (F + 8) * 2.0 ** -23 * ((np.abs(ar) + step) @ np.abs(w2[e]).T)
        k = ids.shape[1]
        y[use] += wt[use, None] * o
        err[use] += np.abs(wt[use, None]) * do + (2 * E + k + 4) * 2.0 ** -24 * np.abs(weights[use]).sum(axis=1)[:, None] * np.abs(o)
    return y, err + 2.0 ** -8 * (np.abs(y) + err) + 1e-38
