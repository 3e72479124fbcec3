"""Pins of the norm oracle (oracle/norm.py): a worked example, invariants and differences of the forward."""
import numpy as np

from oracle import norm as on
from oracle.quant import bf16_to_f32
from oracle.swiglu import round_bf16


def test_worked_example():
    s = round_bf16(np.array([[3.0, 4.0], [1.0, -1.0]]))
    rstd, f = on.norm(s, np.array([2.0, 0.5]), 1e-30)
    np.testing.assert_allclose(rstd, [1 / np.sqrt(12.5), 1.0])
    np.testing.assert_allclose(f, [[6 / np.sqrt(12.5), 2 / np.sqrt(12.5)], [2.0, -0.5]])


def test_residual_sum_rounds_the_fp32_sum():
    a, b = round_bf16(np.array([[1.0, 256.0]])), round_bf16(np.array([[2.0 ** -8, 1.0]]))
    # 1 + 2^-8 is a tie between 1 and 1 + 2^-7: even; 257 is a tie between 256 and 258: even
    np.testing.assert_array_equal(bf16_to_f32(on.residual_sum(a, b)), [[1.0, 256.0]])
    assert on.residual_sum(a, None) is a


def test_normed_rows_have_unit_mean_square():
    rng = np.random.default_rng(1)
    _, f = on.norm(round_bf16(rng.standard_normal((5, 64)) * 7), None, 1e-12)
    np.testing.assert_allclose((f * f).mean(axis=1), 1.0, rtol=1e-9)


def test_backward_against_differences():
    """Central differences of <dh, f(s)> + <dsum, s> in fp64."""
    rng = np.random.default_rng(2)
    R, C, eps = 3, 8, 1e-3
    s, dh, dsum, gamma = (rng.standard_normal(z) for z in ((R, C), (R, C), (R, C), (C,)))

    def loss(s, gamma):
        r = 1 / np.sqrt((s * s).mean(axis=1, keepdims=True) + eps)
        return (dh * s * r * gamma).sum() + (dsum * s).sum()

    rstd = 1 / np.sqrt((s * s).mean(axis=1) + eps)
    dx, dgamma = on.norm_backward(dh, s, rstd, gamma, dsum)
    step = 1e-5
    for r in range(R):
        for c in range(C):
            d = np.zeros((R, C))
            d[r, c] = step
            num = (loss(s + d, gamma) - loss(s - d, gamma)) / (2 * step)
            assert abs(num - dx[r, c]) < 1e-7 * max(1, abs(num))
    for c in range(C):
        d = np.zeros(C)
        d[c] = step
        num = (loss(s, gamma + d) - loss(s, gamma - d)) / (2 * step)
        assert abs(num - dgamma[c]) < 1e-7 * max(1, abs(num))
