"""Pins of the gate oracle (oracle/gate.py): worked examples, invariants, and differences of the forward."""
import numpy as np
import pytest

from oracle import gate as og


def test_worked_choices():
    z = np.array([[1.0, 3.0, 3.0, np.nan], [-np.inf, 0.0, -np.inf, -np.inf], [np.inf, np.inf, 0.0, 1.0]])
    ids, w = og.gate(z, 2, sigmoid=False)
    np.testing.assert_array_equal(ids, [[1, 2], [1, -1], [0, 1]])
    e = np.exp(-2.0)
    np.testing.assert_allclose(w, [[1 / (2 + e)] * 2, [1, 0], [0.5, 0.5]])
    ids, w = og.gate(z, 2, sigmoid=True, bias=[5.0, 0.0, 1.0, 9.0], renorm=True, route_scale=2.0, mask=[1, 0, 1])
    np.testing.assert_array_equal(ids, [[0, 2], [-1, -1], [3, 0]])   # keys 5.73, .95, 1.95; 6, 1, 1.5, 9.73
    a, b = 1 / (1 + np.exp(-1.0)), 1 / (1 + np.exp(-3.0))
    np.testing.assert_allclose(w, [[2 * a / (a + b), 2 * b / (a + b)], [0, 0], [2 * a / (a + 1), 2 / (a + 1)]])


def test_uniform_routing_gives_coef():
    """Uniform scores and uniform counts: f = 1, P = 1 / E, loss = coef, whatever the sequences."""
    E, k, T = 8, 2, 32
    ids = (np.arange(T * k) % E).reshape(T, k)
    for offs in (None, [8, 32], [16, 16, 32]):
        loss, counts, dprob = og.balance(np.zeros((T, E)), ids, 0.3, offs, sigmoid=True)
        S = 1 if offs is None else len(offs)
        empty = 0 if offs is None else sum(b - a == 0 for a, b in zip([0] + offs, offs))
        assert loss == pytest.approx(0.3 * (S - empty) / S)
        assert counts.sum() == T * k
        np.testing.assert_allclose(dprob.sum(axis=1)[dprob.sum(axis=1) > 0].max(), 0.3 / S * E / (8 if S == 2 else
                                                                                              32 if S == 1 else 16))


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("part", ["gate", "loss", "both"])
def test_backward_against_differences(sigmoid, renorm, part):
    rng = np.random.default_rng(3)
    T, E, k = 6, 5, 3
    z = rng.standard_normal((T, E))
    z[1, 2] = -np.inf
    mask = np.array([1, 1, 0, 1, 1, 1])
    offs = [2, 5]
    ids, _ = og.gate(z, k, sigmoid, mask=mask)
    ids[3] = [1, 1, -1]                                    # a repeated choice, a dropped slot
    dw = rng.standard_normal((T, k)) if part != "loss" else None
    _, _, dprob = og.balance(z, ids, 0.7, offs, sigmoid, mask)

    def total(z):
        s, v = og.scores(z, sigmoid), 0.0
        if dw is not None:
            for t in range(T):
                j = [j for j in range(k) if mask[t] and ids[t, j] >= 0]
                w = s[t, ids[t, j]]
                if renorm and len(j):
                    w = w / w.sum()
                v += 1.5 * (w * dw[t, j]).sum()
        if part != "gate":
            p = og.shares(z, sigmoid)
            for i, (lo, hi) in enumerate(og.sequences(offs, T)):
                for t in range(lo, hi):
                    v += 2.0 * mask[t] * (p[t] * dprob[i]).sum()
        return v

    dz, size = og.backward(z, ids, dw, sigmoid, mask, renorm, 1.5, dprob if part != "gate" else None, 2.0, offs)
    for t in range(T):
        for e in range(E):
            if z[t, e] == -np.inf:
                assert dz[t, e] == 0
                continue
            d = np.zeros((T, E))
            d[t, e] = 1e-5
            num = (total(z + d) - total(z - d)) / 2e-5
            assert abs(num - dz[t, e]) < 1e-8 + 1e-7 * abs(num), (t, e)
            assert abs(dz[t, e]) <= size[t, e] * (1 + 1e-12) + 1e-15


def test_loss_is_linear_in_the_shares():
    """<dprob, shares summed over tokens> is the loss: counts are constants of it."""
    rng = np.random.default_rng(4)
    z = rng.standard_normal((40, 6))
    ids, _ = og.gate(z, 2, False)
    loss, _, dprob = og.balance(z, ids, 1.0, [13, 40], False)
    p = og.shares(z, False)
    assert loss == pytest.approx((dprob[0] * p[:13].sum(0)).sum() + (dprob[1] * p[13:].sum(0)).sum())
