"""The integer product for few rows of many groups with short contractions (two waves a workgroup), in both output types."""
import numpy as np
import pytest
import torch

import mxfp8_quantized_moe_amd as fm
from gpu_helpers import note
from mxfp8_quantized_moe_amd import synth
from test_gpu_int8 import check_product

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("M,N,K,E", [(900, 40, 64, 300), (1000, 520, 2048, 64), (400, 1003, 1040, 30), (1500, 648, 272, 100)])
def test_product(M, N, K, E, f32):
    note(f"grouped_mm_scaled INT8 few rows {M}x{N}x{K} of {E} groups f32 {f32}")
    check_product(M, N, K, np.cumsum(synth.random_counts(3, M, E)).tolist(), f32, seed=E)


@pytest.mark.parametrize("M,N,K", [(1, 40, 64), (5, 15, 80), (70, 300, 1040), (3000, 3001, 144)])
def test_one_group_without_offsets(M, N, K):
    """No offsets: one group of all rows, the same bits as with them, in the kernels for few rows and for many."""
    note(f"grouped_mm_scaled INT8 {M}x{N}x{K} without offsets")
    args, out = check_product(M, N, K, [M], False, seed=K)
    args = list(args)
    args[8] = None
    assert torch.equal(fm.grouped_mm_scaled(*args), out)
