"""SwiGLU with its input kept in MXFP8, and the backward from the kept values.

TEST INFRASTRUCTURE ONLY (see the package docstring).

The forward is silu(gate) * up of the bf16 input; what is kept is the input's MX form (``quant.quantize_mx_lastdim``).  The
backward takes the kept values dec(code) * 2^(scale - 127) as gate and up.  All in fp64; ``between`` says which codes an fp32
evaluation may give.
"""
from __future__ import annotations

import numpy as np

from .codec import FMAX, decode, encode_nearest


def kept_values(hq: np.ndarray, hs: np.ndarray) -> np.ndarray:
    return decode(hq, 0) * np.repeat(np.ldexp(1.0, hs.astype(int) - 127), 32, axis=1)


def forward(h: np.ndarray) -> np.ndarray:
    """h fp64 [R, 2F] -> a [R, F]."""
    F = h.shape[1] // 2
    g, u = h[:, :F], h[:, F:]
    return g * u / (1 + np.exp(-g))


def backward(da: np.ndarray, h: np.ndarray):
    """-> (dh [R, 2F], slack [R, 2F]): ten fp32 roundings of the sum's two terms, which may cancel."""
    F = h.shape[1] // 2
    g, u = h[:, :F], h[:, F:]
    s, n = 1 / (1 + np.exp(-g)), 1 / (1 + np.exp(g))
    dh = np.concatenate([da * u * s * (1 + g * n), da * g * s], axis=1)
    mag = np.concatenate([np.abs(da * u * s) * (1 + np.abs(g) * n), np.abs(da * g * s)], axis=1)
    return dh, 10 * 2.0 ** -24 * mag + 1e-38


def between(q: np.ndarray, scale: np.ndarray, v: np.ndarray, slack: np.ndarray, codec: int) -> np.ndarray:
    """Whether each code lies between those of (v - slack) * scale and (v + slack) * scale, one fp32 rounding more each."""
    fmax = float(FMAX[codec])
    s = scale.astype(np.float64)[:, None]
    lo, hi = (v - slack) * s, (v + slack) * s
    lo, hi = lo - 2.0 ** -24 * np.abs(lo), hi + 2.0 ** -24 * np.abs(hi)
    lo, hi = (decode(encode_nearest(np.clip(b, -fmax, fmax), codec), codec) for b in (lo, hi))
    got = decode(q, codec)
    return (lo <= got) & (got <= hi)
