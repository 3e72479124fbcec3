"""Choices between keys score + bias that lie close together: saturated scores, whose differences are 2^-35 and less of a key
with a bias of 3 or 8, far above the 2^-50 or so of a sum in 64 bits.  Ids are whole numbers and must match exactly."""
import numpy as np
import pytest
import torch

import mxfp8_quantized_moe_amd as fm
from oracle import gate as og
from gpu_helpers import DEV, note, host

pytestmark = pytest.mark.gpu


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


@pytest.mark.parametrize("E,k", [(8, 2), (16, 5), (64, 4), (255, 8), (256, 8), (256, 20), (500, 6), (777, 10), (1024, 8)])
@pytest.mark.parametrize("b0", [0.0, 3.0, 8.0, -8.0])
def test_saturated_scores(E, k, b0):
    """Sigmoid scores of logits 24 .. 29.75: steps of the logit by 1/4 move the score by at least 2^-45.3 (e^-29.5 (1 - e^-0.25)),
    the sum with 8 is held to 2^-50.  A row whose larger keys stand at the larger indices, rows in any order, and ties."""
    note(f"moe_gate saturated {E} experts top {k} bias {b0}")
    rng = np.random.default_rng(E + k)
    z = (24 + 0.25 * rng.integers(0, 24, size=(60, E))).astype(np.float32)
    z[::3] = np.sort(z[::3], axis=1)
    bias = np.full(E, b0, np.float32)
    got = host(fm.moe_gate(dev(z), k, fm.GATE_SIGMOID, dev(bias))[0])
    np.testing.assert_array_equal(got, og.gate(z.astype(np.float64), k, True, bias)[0])


@pytest.mark.parametrize("E,k", [(8, 2), (64, 4), (255, 8), (256, 12), (777, 10), (1024, 8)])
@pytest.mark.parametrize("b0", [0.0, 3.0, 8.0])
def test_small_softmax_scores(E, k, b0):
    """One expert holds the row; the others' scores are e^-24 .. e^-29.75 of it."""
    note(f"moe_gate small scores {E} experts top {k} bias {b0}")
    rng = np.random.default_rng(E * 3 + k)
    z = (-24 - 0.25 * rng.integers(0, 24, size=(60, E))).astype(np.float32)
    z[::3] = np.sort(z[::3], axis=1)
    z[np.arange(60), rng.integers(0, E, size=60)] = 0.0
    bias = np.full(E, b0, np.float32)
    got = host(fm.moe_gate(dev(z), k, fm.GATE_SOFTMAX, dev(bias))[0])
    np.testing.assert_array_equal(got, og.gate(z.astype(np.float64), k, False, bias)[0])


def test_named_pairs():
    """Two experts each, the larger key at the higher index."""
    note("moe_gate pairs")
    for b, lo, hi in ((8.0, 24.0, 26.0), (3.0, 26.0, 27.0), (0.0, 30.0, 33.0)):
        ids, _ = fm.moe_gate(torch.tensor([[lo, hi]], device=DEV), 1, fm.GATE_SIGMOID, torch.full((2,), b, device=DEV))
        assert int(ids) == 1, (b, lo, hi)
