"""The integer product with so many rows and columns that the persistent kernel takes it: both of its tiles, one and several
groups, tiles that end inside, every alignment of the output's rows, short contractions, the largest sums, and the bits of the
kernel for few rows."""
import numpy as np
import pytest
import torch

import mxfp8_quantized_moe_amd as fm
from oracle.swiglu import round_bf16
from gpu_helpers import DEV, note, bf16_dev, i32_dev
from test_gpu_int8 import check_product

pytestmark = pytest.mark.gpu

RAGGED12 = [400, 400, 401, 900, 1412, 1412, 1500, 2012, 2300, 2365, 3000, 4980]   # 12 groups: empty ones, 1 and 65 rows
RAGGED40 = np.cumsum(np.arange(40) * 11 % 441).tolist()


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("M,N,K,offs", [
    # one group: 256 x 256 tiles, whole ones and with ends
    (4096, 2304, 128, [4096]), (4100, 2056, 192, [4100]), (4100, 2057, 208, [4000]), (2700, 4098, 144, [2690]),
    # several groups of 512 rows and more each on average: the same tile
    (6000, 1603, 272, [0, 1, 2000, 2129, 5999]), (6144, 1536, 256, [1024, 2048, 4096]),
    # fewer rows a group: 128 x 256 tiles
    (5000, 1501, 176, RAGGED12), (5000, 1504, 400, RAGGED12), (5000, 1538, 1040, RAGGED12),
    (9000, 1000, 336, RAGGED40), (9000, 1003, 128, RAGGED40),
    # fewer columns than the other kernel's smallest tile
    (700, 15, 400, [100, 650]), (1500, 7, 144, [200, 200, 500, 1490]),
])
def test_product(M, N, K, offs, f32):
    note(f"grouped_mm_scaled INT8 persistent {M}x{N}x{K}, {len(offs)} groups, f32 {f32}")
    check_product(M, N, K, offs, f32, seed=M + N + K)


@pytest.mark.parametrize("K", [16, 48, 64, 80, 112, 128, 144, 240, 256, 272, 400, 1040])
@pytest.mark.parametrize("offs", [[2890], [300, 300, 650, 651, 1000, 1400, 1900, 2890]])
def test_contractions(offs, K):
    """Less than a step, one, and up to several rounds of the ring."""
    note(f"grouped_mm_scaled INT8 persistent K {K}, {len(offs)} groups")
    check_product(2900, 2600, K, offs, False, seed=K)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("N", [3000, 3001, 3002, 3004, 3007])
@pytest.mark.parametrize("offs", [[2590], [200, 513, 1000, 1001, 1800, 2590]])
def test_output_rows_at_every_alignment(offs, N, f32):
    note(f"grouped_mm_scaled INT8 persistent N {N}, {len(offs)} groups, f32 {f32}")
    check_product(2600, N, 96, offs, f32, seed=N)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("N", [2056, 2057])
def test_bits_of_the_few_row_kernel(N, f32):
    """A product's rows do not depend on how many others are computed with them, whichever kernel that takes."""
    note(f"grouped_mm_scaled INT8 persistent and few rows N {N} f32 {f32}")
    args, out = check_product(4100, N, 784, [4100], f32, seed=7)
    for rows in (1, 16, 200):
        few = list(args)
        few[1], few[3], few[8], few[10] = args[1][:rows], args[3][:rows], i32_dev([rows]), rows
        assert torch.equal(fm.grouped_mm_scaled(*few, out_dtype=fm.OUT_F32 if f32 else fm.OUT_BF16), out[:rows])


def test_largest_sums():
    """Every product 128 * 128, K the largest multiple of 16 that is taken: 2^31 - 2^18, which fp32 holds exactly."""
    note("grouped_mm_scaled INT8 persistent largest sums")
    M, N, K = 2600, 3600, 131056
    a, b = (torch.full((n, K), -128, dtype=torch.int8, device=DEV) for n in (M, N))
    one = torch.ones(max(M, N), device=DEV)
    out = fm.grouped_mm_scaled(fm.GROUPED_M, a, fm.OPD_INT8, one, b, fm.OPD_INT8, one, fm.SCALE_F32, i32_dev([M]), 1, M, N, K,
                               out_dtype=fm.OUT_F32)
    assert (out == 2.0 ** 31 - 2.0 ** 18).all()


def test_captured():
    """A prompt's linear layer in a graph, replayed on new inputs between eager calls."""
    note("int8 linear of many rows captured")
    rng = np.random.default_rng(4)
    M, N, K = 3000, 2050, 272
    w, ws = fm.quantize_rowwise(bf16_dev(round_bf16(0.02 * rng.standard_normal((N, K)))), codec=fm.INT8)
    xs = [bf16_dev(round_bf16(rng.standard_normal((M, K)))) for _ in range(3)]
    offs = i32_dev([M])

    def linear(x):
        q, s = fm.quantize_rowwise(x, codec=fm.INT8)
        return fm.grouped_mm_scaled(fm.GROUPED_M, q, fm.OPD_INT8, s, w, fm.OPD_INT8, ws, fm.SCALE_F32, offs, 1, M, N, K)

    want = [linear(x) for x in xs]
    x = xs[0].clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = linear(x)
    for i in (0, 1, 2, 1):
        x.copy_(xs[i])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[i])
        linear(xs[0])
