"""Pins of the gate oracle's gradient by differences (oracle/gate.py): against its gradient by the formulas where these keep
their digits, and against 60-digit decimals where they do not."""
from decimal import Decimal as D, getcontext

import numpy as np
import pytest

from oracle import gate as og


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_equals_the_formulas(sigmoid, renorm):
    rng = np.random.default_rng(5)
    T, E, k = 12, 9, 4
    z = rng.standard_normal((T, E))
    z[2, 4:6], z[3] = -np.inf, -np.inf
    mask = np.arange(T) % 5 != 1
    ids, _ = og.gate(z, k, sigmoid, None, mask)
    ids[6, 1] = ids[6, 0]
    dw, dprob = rng.standard_normal((T, k)), rng.random((2, E))
    for d, p in ((dw, None), (None, dprob), (dw, dprob)):
        a, _ = og.backward(z, ids, d, sigmoid, mask, renorm, 1.5, p, 0.5, [5, 11])
        b, size = og.backward_by_differences(z, ids, d, sigmoid, mask, renorm, 1.5, p, 0.5, [5, 11])
        np.testing.assert_allclose(b, a, atol=1e-14, rtol=1e-12)
        assert np.all(np.abs(b) <= size * (1 + 1e-12))


def decimal_gradient(z, ids, dw, sigmoid, renorm, dprob):
    getcontext().prec = 60
    z = [D(float(v)) for v in z]
    s = [1 / (1 + (-v).exp()) if sigmoid else v.exp() for v in z]
    tot = sum(s)
    p = [v / tot for v in s]
    c = [1 - v for v in s] if sigmoid else [D(1)] * len(z)
    out = [D(0)] * len(z)
    if dprob is not None:
        dp = [D(float(v)) for v in dprob]
        dot = sum(a * b for a, b in zip(p, dp))
        out = [a * (b - dot) for a, b in zip(p, dp)]
    if dw is not None:
        dw = [D(float(v)) for v in dw]
        if renorm:
            tot = sum(s[i] for i in ids)
            u = [s[i] / tot for i in ids]
            dot = sum(a * b for a, b in zip(u, dw))
            for i, a, b in zip(ids, u, dw):
                out[i] += a * (b - dot)
        elif sigmoid:
            for i, b in zip(ids, dw):
                out[i] += s[i] * b
        else:
            dot = sum(p[i] * b for i, b in zip(ids, dw))
            out = [o - a * dot for o, a in zip(out, p)]
            for i, b in zip(ids, dw):
                out[i] += p[i] * b
    return np.array([float(o * q) for o, q in zip(out, c)])


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("row", [[20.0, 1.0, -2.0, 0.5], [30.0, 28.0, 29.0, 26.0], [-100.0, -103.0, -101.0, -140.0],
                                 [0.0, -60.0, -61.0, -90.0], [12.0, -40.0, 11.0, 3.0]])
def test_keeps_its_digits(row, sigmoid, renorm):
    rng = np.random.default_rng(6)
    z, ids = np.array([row]), np.array([[0, 2, 3]])
    dw, dprob = rng.standard_normal((1, 3)), rng.random((1, 4))
    for d, p in ((dw, None), (None, dprob), (dw, dprob)):
        got, size = og.backward_by_differences(z, ids, d, sigmoid, None, renorm, 1.0, p)
        want = decimal_gradient(row, ids[0], None if d is None else d[0], sigmoid, renorm, None if p is None else p[0])
        assert np.all(np.abs(got[0] - want) <= 1e-13 * size[0] + 1e-300), (got, want)


def test_shares():
    """On the scale of the row's largest score; none where the sigmoids are 0 in 64 bits, which the formulas give as well."""
    z = np.array([[-100.0, -101.0], [-700.0, -700.0], [-750.0, -750.0], [0.0, -800.0], [-np.inf, -np.inf], [-np.inf, -3.0]])
    a = 1 / (1 + np.exp(-1.0))
    np.testing.assert_allclose(og.loss_shares(z, True), [[a, 1 - a], [0.5, 0.5], [0, 0], [1, 0], [0, 0], [0, 1]])
    np.testing.assert_allclose(og.shares(z, True), og.loss_shares(z, True))
    np.testing.assert_allclose(og.loss_shares(z, False), og.shares(z, False))
