"""Weights beyond the last-level cache's 256 MB, which the kernels for few tokens and few rows read streamed, and weights whose
last experts begin past 2^31 bytes. Most experts are not used, so the 64-bit reference decodes a few."""
import numpy as np
import pytest
import torch

import mxfp8_quantized_moe_amd as fm
from oracle import codec as oc
from oracle import few as of
from oracle.quant import bf16_to_f32
from oracle.swiglu import round_bf16
from gpu_helpers import DEV, note, bf16_dev, i32_dev, host, bf16_bits_to_f64
from test_gpu_int8 import REL16, REL32

pytestmark = pytest.mark.gpu


class Layer:
    """Random codes and scales made on the GPU; `values` decodes the experts asked for."""

    def __init__(self, E, K, F, fmt, seed):
        self.E, self.K, self.F, self.fmt = E, K, F, fmt
        self.g = torch.Generator(DEV).manual_seed(seed)
        self.kw = dict(w_fmt=fm.OPD_INT8 if fmt == "int8" else fm.OPD_E4M3FN,
                       scale_kind={"mx": fm.SCALE_E8M0, "mx_k4": fm.SCALE_E8M0_K4}.get(fmt, fm.SCALE_F32))
        self.w1, self.s1 = self.weights(2 * F, K)
        self.w2, self.s2 = self.weights(K, F)

    def weights(self, rows, cols):
        q = torch.randint(0, 256, (self.E, rows, cols), dtype=torch.uint8, device=DEV, generator=self.g)
        n = self.E * rows
        if self.fmt == "int8":
            return q.view(torch.int8), torch.rand(n, device=DEV, generator=self.g) * 1000 + 2000
        q.bitwise_and_(0xBF)                         # e4m3 values below 2, no NaN among them
        if self.fmt == "fp8":
            return q, torch.rand(n, device=DEV, generator=self.g) * 15 + 15
        shape = fm.mx_k4_shape(n, cols // 32) if self.fmt == "mx_k4" else (n, cols // 32)
        return q, torch.randint(121, 125, shape, dtype=torch.uint8, device=DEV, generator=self.g)

    def values(self, q, s, e):
        c, (rows, cols) = host(q[e]), q.shape[1:]
        v = c.astype(np.float64) if self.fmt == "int8" else oc.decode(c, 0)
        at = slice(e * rows, (e + 1) * rows)
        if not self.fmt.startswith("mx"):
            return v / host(s[at]).astype(np.float64)[:, None]
        code = host(s[:, at]).transpose(1, 0, 2).reshape(rows, -1)[:, :cols // 32] if self.fmt == "mx_k4" else host(s[at])
        return v * np.repeat(np.ldexp(1.0, code.astype(int) - 127), 32, axis=1)

    def check(self, x, ids, w):
        y = fm.moe_few_tokens(bf16_dev(x), i32_dev(ids), torch.from_numpy(w).to(DEV), self.w1, self.s1, self.w2, self.s2, **self.kw)
        got = bf16_bits_to_f64(host(y))
        used = np.unique(ids)
        v1 = np.stack([self.values(self.w1, self.s1, e) for e in used])
        v2 = np.stack([self.values(self.w2, self.s2, e) for e in used])
        ref, bound = of.block(bf16_to_f32(x).astype(np.float64), np.searchsorted(used, ids), w.astype(np.float64), v1, v2)
        bad = ~(np.abs(got - ref) <= bound)
        assert not bad.any(), f"{bad.sum()} of {bad.size} off; worst {np.nanmax(np.abs(got - ref) - bound)} at {np.argwhere(bad)[0]}"


FORMATS = ["fp8", "int8", "mx", "mx_k4"]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("E,K,F,T,k", [
    # short rows: two waves a workgroup from about 512 workgroups on, four below
    (96, 1024, 1024, 1, 4), (96, 1024, 1024, 4, 4), (96, 1024, 1024, 8, 4), (96, 1024, 1024, 16, 4), (96, 1024, 1024, 30, 4),
    (96, 1024, 1024, 64, 4), (96, 1024, 992, 1, 16),
    # long rows in W1 and short ones in W2, long rows in both
    (12, 4096, 2048, 5, 4), (12, 4096, 2048, 40, 3), (6, 4096, 4160, 3, 2), (6, 4096, 4160, 30, 2), (6, 4160, 4096, 64, 2),
])
def test_moe_few_tokens(E, K, F, T, k, fmt):
    note(f"moe_few_tokens streamed {fmt} E {E} K {K} F {F} T {T} topk {k}")
    assert 3 * E * K * F > 256 << 20
    rng = np.random.default_rng(E + T)
    ids = np.tile(rng.permutation(E)[:k], (T, 1)).astype(np.int32)      # every token at the same experts
    x = round_bf16(rng.standard_normal((T, K)))
    Layer(E, K, F, fmt, T).check(x, ids, rng.standard_normal((T, k)).astype(np.float32))


@pytest.mark.parametrize("fmt", FORMATS)
def test_moe_few_tokens_past_2_31(fmt):
    note(f"moe_few_tokens {fmt}, experts past 2^31 bytes")
    E, K, F = 520, 2048, 2048
    assert (E - 1) * K * F > 1 << 31
    rng = np.random.default_rng(2)
    ids = np.array([[519, 300], [519, 0], [300, 519]], np.int32)
    Layer(E, K, F, fmt, 9).check(round_bf16(rng.standard_normal((3, K))), ids, rng.standard_normal((3, 2)).astype(np.float32))


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("M,N,K,offs", [
    # long rows: four waves, 32 columns a workgroup and, beyond 32 rows, 64
    (3, 17000, 16384, [3]), (8, 17003, 16384, [8]), (30, 17000, 16384, [30]), (40, 17001, 16384, [40]), (60, 17000, 16368, [60]),
    # short rows: two waves
    (2, 140000, 2048, [2]), (12, 140001, 2032, [12]),
    # groups past 2^31 bytes
    (9, 2048, 2048, [2] * 260 + [3] * 259 + [9]), (40, 2050, 2048, [5] * 400 + [6] * 120 + [40]),
])
def test_integer_product(M, N, K, offs, f32):
    note(f"grouped_mm_scaled INT8 streamed {M}x{N}x{K}, {len(offs)} groups, f32 {f32}")
    E = len(offs)
    assert E * N * K > 256 << 20
    g = torch.Generator(DEV).manual_seed(M)
    draw = lambda *shape: torch.randint(-128, 128, shape, dtype=torch.int8, device=DEV, generator=g)
    a, b = draw(M, K), draw(E, N, K)
    sa, sb = torch.rand(M, device=DEV, generator=g) * 90 + 0.5, torch.rand(E, N, device=DEV, generator=g) * 9000 + 100
    out = fm.grouped_mm_scaled(fm.GROUPED_M, a, fm.OPD_INT8, sa, b, fm.OPD_INT8, sb, fm.SCALE_F32, i32_dev(offs), E, M, N, K,
                               out_dtype=fm.OUT_F32 if f32 else fm.OUT_BF16)
    lo = 0
    for e, hi in enumerate(offs):
        if hi > lo:
            s = torch.mm(a[lo:hi].double(), b[e].double().t().contiguous())      # whole numbers below 2^53: exact
            ref = s / (sa[lo:hi, None].double() * sb[e].double())
            off = (out[lo:hi].double() - ref).abs() - (REL32 if f32 else REL16) * ref.abs()
            assert (off <= 0).all(), float(off.max())
        lo = max(lo, hi)
