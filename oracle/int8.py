"""Symmetric 8-bit integer quantization and the product of its codes.

TEST INFRASTRUCTURE ONLY (see the package docstring).

The rowwise recipe with fmax 127: s = fp32(127 * fp32(1 / max(amax, 1e-12))), y =
clamp(fp32(x * s), -127, 127), q = the whole number nearest to y, ties to even.
The product of two such operands sums whole numbers: exact in fp64 below 2^53.
"""
from __future__ import annotations

import numpy as np

from .gemm import group_bounds
from .quant import EPS, bf16_to_f32

FMAX = np.float32(127)


def quantize_rows_f32(f: np.ndarray):
    """fp32 rows -> (codes int8 [R, C], scale f32 [R])."""
    f = np.asarray(f, np.float32)
    amax = np.abs(f).max(axis=1) if f.shape[1] else np.zeros(f.shape[0], np.float32)
    scale = FMAX * (np.float32(1) / np.maximum(amax, EPS))
    y = np.clip(f * scale[:, None], -FMAX, FMAX)
    return np.rint(y).astype(np.int8), scale


def quantize_rowwise(x_bits: np.ndarray):
    """bf16 rows -> (codes int8 [R, C], scale f32 [R])."""
    return quantize_rows_f32(bf16_to_f32(x_bits))


def mm_grouped_m(a: np.ndarray, sa: np.ndarray, b: np.ndarray, sb: np.ndarray, offs) -> np.ndarray:
    """a int8 [M, K], b int8 [E, N, K] -> fp64 [M, N]: sums of products over the scales; NaN in rows of no group."""
    out = np.full((a.shape[0], b.shape[1]), np.nan)
    for e, (lo, hi) in enumerate(zip(*group_bounds(offs, a.shape[0]))):
        acc = a[lo:hi].astype(np.float64) @ b[e].astype(np.float64).T   # whole numbers below 2^53: exact
        out[lo:hi] = acc / (sa[lo:hi, None].astype(np.float64) * sb[e][None].astype(np.float64))
    return out
