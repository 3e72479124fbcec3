"""Gradients of tokens of which one expert holds almost everything: a softmax score, a share of the loss or a renormalised
weight within 2^-24 and less of 1.  The gradient is then the small rest's, each to its own digits, against the gradient by
differences (oracle/gate.py).

Tolerances as in test_gpu_gate_confident.py.  With a u above a half, x_i - x_top costs one rounding: the terms u_j (x_j - x_top)
are within e + 4 u of u_j (|x_j| + |x_top|), their sum 22 u of additions more.  For i = top these are the size; for another i
the size holds u_i (|x_i| + |x_top|) / 2, and twice the sum's error comes on top: 6 e + 60 u = (36 X + 240) u, and (3 X + 6) u
of a sigmoid's complement: below (40 X + 300) u size."""
import numpy as np
import pytest

from oracle import gate as og
from gpu_helpers import note
from test_gpu_gate_confident import check, device_logits

pytestmark = pytest.mark.gpu

SIZES = [(2, 1), (4, 2), (7, 3), (16, 1), (40, 4), (64, 6), (128, 2), (255, 8), (256, 8), (500, 3), (1024, 12)]


@pytest.mark.parametrize("E,k", SIZES)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_one_expert_holds_the_token(E, k, dtype, sigmoid):
    """One expert 1 .. 45 above the others (softmax), or at -2 .. 10 over others that are as far below 0 (sigmoid)."""
    rng = np.random.default_rng(E * 5 + k)
    T = 46
    z = rng.uniform(-1, 0, size=(T, E)) - np.arange(T)[:, None]
    z[np.arange(T), rng.integers(0, E, size=T)] = rng.uniform(-2, 10, size=T) if sigmoid else 0.5
    z = z[rng.permutation(T)]                                # confident tokens beside others in a wave
    zd, z = device_logits(z, dtype)
    ids, _ = og.gate(z, k, sigmoid)
    dw = rng.standard_normal((T, k)).astype(np.float32)
    dprob = rng.random((2, E)).astype(np.float32)
    for renorm in (False, True):
        for a, b in ((dw, None), (None, dprob), (dw, dprob)):
            check(z, zd, ids, a, b, sigmoid, renorm, [13, T],
                  f"dominant {E} top {k} {dtype} sigmoid {sigmoid} renorm {renorm} {a is None} {b is None}")


@pytest.mark.parametrize("sigmoid", [False, True])
def test_two_experts_hold_the_token(sigmoid):
    """Two equal scores of a half each, and two nearly so."""
    note("two experts")
    rng = np.random.default_rng(9)
    z = np.full((20, 16), -30.0)
    z[:, 3], z[:, 11] = 0.0, np.where(np.arange(20) % 2, 0.0, 1e-6)
    zd, z = device_logits(z, "f32")
    ids, _ = og.gate(z, 4, sigmoid)
    dw, dprob = rng.standard_normal((20, 4)).astype(np.float32), rng.random((2, 16)).astype(np.float32)
    for renorm in (False, True):
        for a, b in ((dw, None), (None, dprob), (dw, dprob)):
            check(z, zd, ids, a, b, sigmoid, renorm, [5, 20], f"two experts sigmoid {sigmoid} renorm {renorm}")
