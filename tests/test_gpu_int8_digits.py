"""The integer product's fp32 outputs have the digits of two divisions, in the kernels for few rows and for many alike."""
import numpy as np
import pytest
import torch

import mxfp8_quantized_moe_amd as fm
from gpu_helpers import DEV, note, i32_dev, host

pytestmark = pytest.mark.gpu

# The exact sum is rounded to fp32 and divided twice: three half steps, and what a quotient formed from a reciprocal and its
# error adds to each (under 2^-22 of a half step).
THREE = 3.01 * 2.0 ** -24


@pytest.mark.parametrize("M,N,K,offs", [
    (16, 3001, 1040, [16]), (40, 260, 64, [7, 40]), (500, 1999, 80, [130, 130, 500]), (12, 15, 4096, [12]),
    (2600, 3001, 96, [2600]), (2600, 3008, 208, [2600]), (4000, 2050, 144, [300, 301, 900, 1500, 1900, 2400, 3000, 4000]),
])
def test_three_half_steps(M, N, K, offs):
    note(f"grouped_mm_scaled INT8 fp32 digits {M}x{N}x{K}, {len(offs)} groups")
    rng = np.random.default_rng(M + N)
    E = len(offs)
    a, b = rng.integers(-127, 128, (M, K)).astype(np.int8), rng.integers(-127, 128, (E, N, K)).astype(np.int8)
    sa, sb = (np.exp2(rng.uniform(-20, 40, n)).astype(np.float32) for n in (M, (E, N)))
    dev = lambda v: torch.from_numpy(v).to(DEV)
    got = host(fm.grouped_mm_scaled(fm.GROUPED_M, dev(a), fm.OPD_INT8, dev(sa), dev(b), fm.OPD_INT8, dev(sb), fm.SCALE_F32,
                                    i32_dev(offs), E, M, N, K, out_dtype=fm.OUT_F32)).astype(np.float64)
    lo = 0
    for e, hi in enumerate(offs):
        ref = a[lo:hi].astype(np.float64) @ b[e].astype(np.float64).T / (sa[lo:hi, None].astype(np.float64) * sb[e].astype(np.float64))
        off = np.abs(got[lo:hi] - ref) - THREE * np.abs(ref)
        assert (off <= 0).all(), f"group {e}: {(off > 0).mean():.2e} of the outputs off"
        lo = hi


@pytest.mark.parametrize("M,N", [(20, 300), (2600, 3001)])
def test_an_infinite_row(M, N):
    """A token with an infinity has the scale 0: its own outputs are not finite, the others' are as without it."""
    note(f"grouped_mm_scaled INT8 fp32 {M}x{N}, an infinite row")
    K = 96
    g = torch.Generator(DEV).manual_seed(1)
    x = torch.randn(M, K, device=DEV, generator=g).to(torch.bfloat16)
    w, ws = fm.quantize_rowwise(torch.randn(N, K, device=DEV, generator=g).to(torch.bfloat16), codec=fm.INT8)

    def linear(x):
        q, s = fm.quantize_rowwise(x, codec=fm.INT8)
        return fm.grouped_mm_scaled(fm.GROUPED_M, q, fm.OPD_INT8, s, w, fm.OPD_INT8, ws, fm.SCALE_F32, None, 1, M, N, K,
                                    out_dtype=fm.OUT_F32)

    ref = linear(x)
    x[7, 3] = float("inf")
    got = linear(x)
    assert not torch.isfinite(got[7]).any()
    keep = torch.arange(M, device=DEV) != 7
    assert torch.equal(got[keep], ref[keep])


@pytest.mark.parametrize("M,N", [(16, 40), (2600, 3001)])
def test_beyond_fp32(M, N):
    """Quotients beyond fp32 are infinities of their sign, as division makes them, in each order of overflow; a sum of 0 over
    such scales is 0; scales of infinity give 0."""
    note(f"grouped_mm_scaled INT8 fp32 {M}x{N} beyond the range")
    K = 16
    a, b = torch.ones(M, K, dtype=torch.int8, device=DEV), torch.ones(N, K, dtype=torch.int8, device=DEV)
    a[::3] = -1
    a[2::3, ::2] = -1                      # sums -16, 16, 0
    sa, sb = torch.ones(M, device=DEV), torch.ones(N, device=DEV)
    sa[3:], sb[5:] = 2.0 ** -125, 2.0 ** -100     # the second quotient overflows from row 3 and column 5 on
    sa[9:] = 2.0 ** -126                          # 16 / 2^-126 does not fit in fp32: the first quotient overflows
    sb[12], sa[15] = float("inf"), 0.0
    out = fm.grouped_mm_scaled(fm.GROUPED_M, a, fm.OPD_INT8, sa, b, fm.OPD_INT8, sb, fm.SCALE_F32, None, 1, M, N, K,
                               out_dtype=fm.OUT_F32)
    # as quotients, in fp32: the sum over the row's scale, and that over the column's
    sums = (a.double() @ b.double().t().contiguous()).float()
    ref = (sums / sa[:, None]) / sb
    finite = torch.isfinite(ref)
    assert torch.equal(out[finite], ref[finite])              # powers of two: exact
    assert torch.equal(torch.isnan(out), torch.isnan(ref))
    inf = torch.isinf(ref)
    assert inf.any() and torch.equal(out[inf], ref[inf])
