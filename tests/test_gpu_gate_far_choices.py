"""Renormalised weights of choices whose scores are all below the fp32 range (a bias that chooses experts far below the row's
largest logit; sigmoid logits of -90 and less): their ratios, and the gradient through them.

Tolerances as in test_gpu_gate.py and test_gpu_gate_confident.py: a weight within 2 (6 X + 30) u, X the distances among the
chosen logits (a sigmoid's at most 90), values below 2^-126 may be flushed."""
import numpy as np
import pytest
import torch

import mxfp8_quantized_moe_amd as fm
from oracle import gate as og
from gpu_helpers import DEV, note, host, i32_dev

pytestmark = pytest.mark.gpu

U, TINY = 2.0 ** -24, 2.0 ** -126
LOWEST = float(np.finfo(np.float32).min)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def check(z, ids, w, sigmoid, scale, what):
    """Weights and gradient of the choices `ids` [T, k] (all eligible) of fp64 logits z."""
    T, k = ids.shape
    zc = np.take_along_axis(z, ids, axis=1)
    u = og.parts_of_one(zc, sigmoid)
    X = float(np.minimum(np.abs(zc.max(axis=1, keepdims=True) - zc), 90).max())
    tol = 2 * (6 * X + 30 + (24 if sigmoid else 0)) * U      # a sigmoid's own reciprocal and second exponential
    got = host(w)
    assert np.all(np.abs(got - scale * u) <= scale * (tol * u + 4 * TINY)), f"{what}: {got[0]} want {scale * u[0]}"
    rng = np.random.default_rng(3)
    dw = rng.standard_normal((T, k)).astype(np.float32)
    dz, size = og.backward_by_differences(z, ids, dw, sigmoid, None, True, scale)
    g = host(fm.moe_gate_backward(dev(z.astype(np.float32)), i32_dev(ids), dev(dw), int(sigmoid), None, True, scale))
    mag = np.zeros_like(size)                                # terms before any of them cancel
    np.add.at(mag, (np.arange(T)[:, None], ids), scale * u * (np.abs(dw) + (np.abs(dw) * u).sum(axis=1, keepdims=True)))
    assert np.all(np.abs(g - dz) <= (40 * X + 300) * U * mag + 8 * TINY * scale * 10), what


@pytest.mark.parametrize("E,k", [(4, 1), (16, 3), (64, 6), (100, 20), (255, 8), (256, 8), (1024, 12)])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("depth", [50.0, 88.0, 100.0, 150.0, 1000.0, 1e30])
def test_a_bias_chooses_far_experts(E, k, sigmoid, depth):
    """k experts around -depth, chosen by a bias in the bias's order; the others around 0."""
    note(f"moe_gate far choices {E} top {k} sigmoid {sigmoid} depth {depth}")
    rng = np.random.default_rng(E + k)
    T = 30
    z = rng.standard_normal((T, E)).astype(np.float32)
    far = rng.permutation(E)[:k]
    z[:, far] = (-depth + 2 * rng.standard_normal((T, k))).astype(np.float32)
    bias = np.zeros(E, np.float32)
    bias[far] = 8 + np.arange(k, 0, -1)
    ids, w = fm.moe_gate(dev(z), k, int(sigmoid), dev(bias), None, True, 2.5)
    np.testing.assert_array_equal(host(ids), np.broadcast_to(far, (T, k)))
    check(z.astype(np.float64), host(ids).astype(np.int64), w, sigmoid, 2.5, f"{E} top {k} depth {depth}")
    if k == 1:
        assert bool((w == 2.5).all())
    both = fm.moe_gate_balance(dev(z), k, 0.1, None, int(sigmoid), dev(bias), None, True, 2.5)
    assert torch.equal(both[0], ids)
    assert bool(((both[1] - w).abs() <= 16 * U * w).all())


@pytest.mark.parametrize("level", [-80.0, -87.5, -90.0, -100.0, -500.0, LOWEST])
def test_low_sigmoid_rows(level):
    """Whole rows of low logits, no bias: weights that sum to the scale, a single choice exactly the scale."""
    note(f"moe_gate low sigmoid rows {level}")
    rng = np.random.default_rng(7)
    z = np.full((20, 32), level, np.float32)
    if level > -1e3:
        z += rng.uniform(0, 3, size=z.shape).astype(np.float32)
    for k in (1, 4, 32):
        ids, w = fm.moe_gate(dev(z), k, fm.GATE_SIGMOID, renormalize=True)
        np.testing.assert_array_equal(host(ids), og.gate(z.astype(np.float64), k, True)[0])
        check(z.astype(np.float64), host(ids).astype(np.int64), w, True, 1.0, f"level {level} top {k}")
        if k == 1:
            assert bool((w == 1).all())


def test_choices_of_the_lowest_value():
    """Softmax rows whose chosen experts are masked out by the type's lowest value: equal weights."""
    note("moe_gate lowest choices")
    z = np.random.default_rng(8).standard_normal((9, 16)).astype(np.float32)
    z[:, 4:8] = LOWEST
    bias = np.zeros(16, np.float32)
    bias[4:8] = 9.0
    for score in (0, 1):
        ids, w = fm.moe_gate(dev(z), 4, score, dev(bias), renormalize=True)
        np.testing.assert_array_equal(host(ids), np.tile(np.arange(4, 8), (9, 1)))
        assert bool((w == 0.25).all())
