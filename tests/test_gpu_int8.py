"""8-bit integers with a scale for each token and each channel: quantizers bit for bit, products within the roundings that
the contract names."""
import numpy as np
import pytest
import torch

import mxfp8_quantized_moe_amd as fm
from mxfp8_quantized_moe_amd import synth
from oracle import int8 as oi
from oracle.quant import bf16_to_f32
from oracle.swiglu import round_bf16
from gpu_helpers import DEV, note, bf16_dev, i32_dev, host, bf16_bits_to_f64, assert_bytes_equal, assert_f32_bits_equal

pytestmark = pytest.mark.gpu

INT8 = fm.INT8
PAD_SCALE = np.float32(127) * (np.float32(1) / np.float32(1e-12))


def rows(rng, R, C):
    x = rng.standard_normal((R, C)) * np.where(rng.random((R, C)) < 0.01, 30, 1)
    if R > 2:
        x[R // 2] = 0                                   # a row of zeros
        x[R // 3] *= 1e-20                              # a row below the floor of the scale
    return round_bf16(x)


@pytest.mark.parametrize("R,C,pad", [(1, 8, 0), (7, 24, 8), (130, 520, 0), (33, 2056, 40), (16, 4096, 0), (5, 16392, 0)])
def test_quantize_rowwise(R, C, pad):
    note(f"quantize_rowwise INT8 {R}x{C} pad {pad}")
    x = rows(np.random.default_rng(R + C), R, C + pad)
    q, s = fm.quantize_rowwise(bf16_dev(x)[:, :C], codec=INT8)
    assert q.dtype == torch.int8
    rq, rs = oi.quantize_rowwise(x[:, :C])
    assert_f32_bits_equal(host(s), rs, "scale")
    assert_bytes_equal(host(q), rq, "codes")


def test_ties():
    note("quantize_rowwise INT8 ties")
    x = round_bf16(np.tile(np.array([[127, 0.5, 1.5, 2.5, -0.5, -1.5, -2.5, 126.5]]), (3, 5)))
    q, s = fm.quantize_rowwise(bf16_dev(x), codec=INT8)
    assert host(q)[0, :8].tolist() == [127, 0, 2, 2, 0, -2, -2, 126]


@pytest.mark.parametrize("R,F", [(3, 8), (50, 336), (17, 1408), (4, 8200)])
def test_swiglu(R, F):
    note(f"swiglu_quantize_rowwise INT8 {R}x{F}")
    h1 = rows(np.random.default_rng(F), R, 2 * F)
    a2, q, s = fm.swiglu_quantize_rowwise(bf16_dev(h1), codec=INT8)
    ref = fm.swiglu_quantize_rowwise(bf16_dev(h1))[0]
    assert_bytes_equal(host(a2), host(ref), "a2")
    rq, rs = oi.quantize_rowwise(host(a2))
    assert_f32_bits_equal(host(s), rs, "scale")
    assert_bytes_equal(host(q), rq, "codes")


@pytest.mark.parametrize("C", [64, 2048])
def test_gathers(C):
    note(f"moe_permute_rowwise / _quantized INT8 C {C}")
    rng = np.random.default_rng(C)
    T, k, E = 37, 3, 5
    x = rows(rng, T, C)
    ids = i32_dev(rng.integers(-1, E, (T, k)))
    _, _, _, src = fm.moe_route(ids, E, 16)
    sl = host(src)
    xg, qg, sg = fm.moe_permute_rowwise(bf16_dev(x), src, k, codec=INT8)
    q, s = fm.quantize_rowwise(bf16_dev(x), codec=INT8)
    qg2, sg2 = fm.moe_permute_quantized(q, s, src, k, codec=INT8)
    rq, rs = oi.quantize_rowwise(x)
    want = np.where((sl >= 0)[:, None], rq[np.maximum(sl, 0) // k], 0).astype(np.int8)
    wants = np.where(sl >= 0, rs[np.maximum(sl, 0) // k], PAD_SCALE).astype(np.float32)
    for name, a, b in (("rowwise", qg, sg), ("quantized", qg2, sg2)):
        assert_bytes_equal(host(a), want, name)
        assert_f32_bits_equal(host(b), wants, name)


@pytest.mark.parametrize("R,C", [(1, 8), (21, 256), (300, 2056), (16, 7168), (9, 12296)])
def test_norm(R, C):
    note(f"rmsnorm_quantize_rowwise INT8 {R}x{C}")
    rng = np.random.default_rng(R + C)
    x, gamma = round_bf16(rng.standard_normal((R, C))), round_bf16(1 + 0.2 * rng.standard_normal(C))
    h, q, s, rstd, _ = fm.rmsnorm_quantize_rowwise(bf16_dev(x), bf16_dev(gamma), 1e-6, codec=INT8)
    f = (bf16_to_f32(x) * bf16_to_f32(gamma)) * host(rstd)[:, None]
    rq, rs = oi.quantize_rows_f32(f)
    assert q.dtype == torch.int8
    assert_f32_bits_equal(host(s), rs, "scale")
    assert_bytes_equal(host(q), rq, "codes")
    ref = fm.rmsnorm_quantize_rowwise(bf16_dev(x), bf16_dev(gamma), 1e-6, codes=False)
    assert_bytes_equal(host(h), host(ref[0]), "h")


# The sum is exact; fp32 then rounds the integer, two reciprocals and two products: (1 + 2^-24)^5 - 1 < 5.01 * 2^-24 of the
# value, and the bf16 output half a step more (2^-8 of the value at most).
REL32, REL16 = 5.01 * 2.0 ** -24, 2.0 ** -8 + 5.1 * 2.0 ** -24


def check_product(M, N, K, offs, f32, seed=0, a=None, b=None):
    rng = np.random.default_rng(seed)
    E = len(offs)
    a = rng.integers(-127, 128, (M, K)).astype(np.int8) if a is None else a
    b = rng.integers(-127, 128, (E, N, K)).astype(np.int8) if b is None else b
    sa, sb = rng.uniform(0.5, 90, M).astype(np.float32), rng.uniform(100, 9000, (E, N)).astype(np.float32)
    ref = oi.mm_grouped_m(a, sa, b, sb, np.asarray(offs, np.int32))
    out = torch.full((M, N), -7.0, dtype=torch.float32 if f32 else torch.bfloat16, device=DEV)
    dev = lambda v: torch.from_numpy(np.ascontiguousarray(v)).to(DEV)
    args = (fm.GROUPED_M, dev(a), fm.OPD_INT8, dev(sa), dev(b), fm.OPD_INT8, dev(sb), fm.SCALE_F32, i32_dev(offs), E, M, N, K)
    fm.grouped_mm_scaled(*args, out=out, out_dtype=fm.OUT_F32 if f32 else fm.OUT_BF16)
    got = host(out)
    got = got.astype(np.float64) if f32 else bf16_bits_to_f64(got)
    outside = np.isnan(ref)
    assert (got[outside] == -7.0).all(), "rows of no group were written"
    err = np.abs(got - ref)[~outside]
    lim = (REL32 if f32 else REL16) * np.abs(ref)[~outside]
    assert (err <= lim).all(), f"worst {np.max(err - lim)}"
    again = fm.grouped_mm_scaled(*args, out_dtype=fm.OUT_F32 if f32 else fm.OUT_BF16)
    assert (again[~torch.from_numpy(outside.all(1))] == out[~torch.from_numpy(outside.all(1))]).all()
    return args, out


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("M,N,K,offs", [
    (1, 1, 16, [1]), (1, 40, 4096, [1]), (16, 300, 1040, [16]), (33, 257, 128, [33]), (64, 512, 2064, [64]),
    (65, 129, 144, [65]), (300, 513, 272, [300]), (700, 264, 400, [700]),
    (77, 96, 192, [10, 10, 9, 60, 60]), (500, 270, 176, [-3, 130, 131, 600, 480]), (40, 64, 64, [0, 0]),
    (1200, 130, 320, [600, 1150]), (2, 24, 32, [1, 2]), (5000, 48, 64, [20, 5000]),
    (150, 67, 208, [0, 1, 140, 150]), (90, 100, 4112, [70, 90]), (3, 33, 1008, [3]), (260, 72, 96, [3, 5, 260]), (24, 31, 64, [24]),
    (7, 14336, 64, [7]), (200, 14336, 64, [200]),
    # few columns, short of a tile's width
    (70, 16, 80, [70]), (33, 17, 1040, [33]), (40, 24, 192, [3, 40]), (5, 31, 272, [2, 2, 5]), (100, 15, 144, [100]), (90, 40, 528, [90]),
    # a contraction shorter than a step, one step, and little more
    (50, 40, 16, [50]), (20, 40, 16, [20]), (3, 40, 16, [3]), (60, 80, 48, [60]), (60, 80, 80, [60]), (200, 4096, 272, [200]),
    # the persistent kernel: rows of the output that do not begin on 16 bytes, tiles that N or a group ends in
    # (sizes that the kernel for few rows takes by now; the persistent one's are in test_gpu_int8_persistent.py)
    (1200, 2503, 320, [600, 1150]), (700, 4099, 208, [650]), (4200, 779, 176, [1000, 1000, 4100]), (900, 3586, 144, [5, 900]),
])
def test_product(M, N, K, offs, f32):
    note(f"grouped_mm_scaled INT8 {M}x{N}x{K} offs {offs} f32 {f32}")
    check_product(M, N, K, offs, f32, seed=M + N + K)


def test_product_many_groups():
    rng = np.random.default_rng(3)
    offs = np.cumsum(synth.random_counts(3, 900, 300))
    note("grouped_mm_scaled INT8 300 groups")
    check_product(900, 40, 64, offs.tolist(), True, seed=5)


@pytest.mark.parametrize("M", [3, 200])
def test_product_largest_sums(M):
    """Every product 128 * 128, K the largest multiple of 16 that is taken: the sum is 2^31 - 2^18."""
    note(f"grouped_mm_scaled INT8 largest sums M {M}")
    K = 131056
    a, b = np.full((M, K), -128, np.int8), np.full((1, 5, K), -128, np.int8)
    check_product(M, 5, K, [M], True, a=a, b=b)
    b[:] = 127
    check_product(M, 5, K, [M], True, a=a, b=b)


def test_product_empty():
    note("grouped_mm_scaled INT8 no rows, no contraction")
    e = torch.empty(0, dtype=torch.int8, device=DEV)
    s = torch.ones(8, device=DEV)
    w = torch.ones(8, 16, dtype=torch.int8, device=DEV)
    out = fm.grouped_mm_scaled(fm.GROUPED_M, e, fm.OPD_INT8, s, w, fm.OPD_INT8, s, fm.SCALE_F32, i32_dev([0]), 1, 0, 8, 16)
    assert out.shape == (0, 8)
    out = fm.grouped_mm_scaled(fm.GROUPED_M, e, fm.OPD_INT8, s, e, fm.OPD_INT8, s, fm.SCALE_F32, i32_dev([4]), 1, 4, 8, 0)
    assert (host(out) == 0).all()


def test_product_captured_and_on_a_stream():
    """A graph of the quantizer and the product, replayed on new inputs beside eager calls on another stream."""
    note("int8 linear captured")
    rng = np.random.default_rng(9)
    M, N, K = 24, 200, 512
    w, ws = fm.quantize_rowwise(bf16_dev(round_bf16(0.02 * rng.standard_normal((N, K)))), codec=INT8)
    xs = [bf16_dev(round_bf16(rng.standard_normal((M, K)))) for _ in range(3)]
    offs = i32_dev([M])

    def linear(x):
        q, s = fm.quantize_rowwise(x, codec=INT8)
        return fm.grouped_mm_scaled(fm.GROUPED_M, q, fm.OPD_INT8, s, w, fm.OPD_INT8, ws, fm.SCALE_F32, offs, 1, M, N, K)

    x = xs[0].clone()
    linear(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        linear(x)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = linear(x)
    for v in xs + xs:
        x.copy_(v)
        g.replay()
        with torch.cuda.stream(side):
            other = linear(xs[1])
        torch.cuda.synchronize()
        assert torch.equal(y, linear(v)) and torch.equal(other, linear(xs[1]))
