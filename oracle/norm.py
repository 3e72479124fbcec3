"""The root-mean-square norm with the residual's addition, and its backward.

TEST INFRASTRUCTURE ONLY (see the package docstring).

s = bf16(x + residual) (one fp32 sum), rstd = 1 / sqrt(mean(s^2) + eps),
f = s * gamma * rstd; h is f rounded to bf16 and the codes quantize f itself
(not h).  Everything after s is computed in fp64 here; how far the fp32
kernels may be from it is derived in the tests.  Backward, from the quotient
rule with n = s * rstd and g = dh * gamma:
  d s = rstd * (g - n * mean(g * n)) + dsum,   d gamma = sum over rows dh * n.
"""
from __future__ import annotations

import numpy as np

from .quant import bf16_to_f32
from .swiglu import round_bf16


def residual_sum(x_bits: np.ndarray, res_bits: np.ndarray | None) -> np.ndarray:
    """bf16 bits of x + residual: the exact sum rounded to fp32, then to bf16."""
    if res_bits is None:
        return x_bits
    return round_bf16((bf16_to_f32(x_bits) + bf16_to_f32(res_bits)).astype(np.float64))


def norm(s_bits: np.ndarray, gamma: np.ndarray | None, eps: float):
    """-> (rstd [R], f [R, C]) in fp64."""
    s = bf16_to_f32(s_bits).astype(np.float64)
    rstd = 1.0 / np.sqrt((s * s).sum(axis=1) / s.shape[1] + float(np.float32(eps)))
    f = s * rstd[:, None]
    return rstd, f if gamma is None else f * np.asarray(gamma, np.float64)


def norm_backward(dh: np.ndarray, s: np.ndarray, rstd: np.ndarray, gamma: np.ndarray | None,
                  dsum: np.ndarray | None):
    """fp64 inputs -> (dx [R, C], dgamma [C])."""
    n = s * rstd[:, None]
    g = dh if gamma is None else dh * gamma
    dx = rstd[:, None] * (g - n * (g * n).mean(axis=1, keepdims=True))
    return (dx if dsum is None else dx + dsum), (dh * n).sum(axis=0)
