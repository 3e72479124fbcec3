"""The kept SwiGLU oracle against differences and scalar arithmetic."""
import math

import numpy as np
import pytest

from oracle import codec as oc
from oracle import quant as oq
from oracle import saved as os_
from oracle.swiglu import round_bf16


def test_backward_is_the_derivative():
    rng = np.random.default_rng(0)
    h, da = 3 * rng.standard_normal((4, 64)), rng.standard_normal((4, 32))
    dh, slack = os_.backward(da, h)
    eps = 1e-5
    for r, c in [(0, 0), (1, 17), (2, 31), (3, 32), (0, 50), (1, 63)]:
        hp, hm = h.copy(), h.copy()
        hp[r, c] += eps
        hm[r, c] -= eps
        d = ((os_.forward(hp) - os_.forward(hm)) * da).sum() / (2 * eps)
        assert dh[r, c] == pytest.approx(d, rel=1e-7, abs=1e-9)
    wrong = np.concatenate([dh[:, 32:], dh[:, :32]], axis=1)     # gate and up exchanged
    assert (np.abs(wrong - dh) > slack).mean() > 0.9


def test_kept_values_by_scalars():
    rng = np.random.default_rng(1)
    x = round_bf16(rng.standard_normal((3, 96)) * 10.0 ** rng.integers(-6, 3, (3, 1)))
    for rule in (0, 1):
        q, s = oq.quantize_mx_lastdim(x, rule)[:2]
        v = os_.kept_values(q, s)
        table = oc.decode_table(0)
        for r in range(3):
            for c in range(96):
                assert v[r, c] == math.ldexp(float(table[q[r, c]]), int(s[r, c // 32]) - 127)
        # within e4m3's half step of the block's scale, and the FLOOR rule's clamp (at most 1/8 of the value)
        f = oq.bf16_to_f32(x).astype(np.float64)
        step = np.repeat(np.ldexp(2.0 ** -10, s.astype(int) - 127), 32, axis=1)
        assert (np.abs(v - f) <= np.maximum((2.0 ** -4 if rule else 2.0 ** -3) * np.abs(f), step)).all()


@pytest.mark.parametrize("codec", [0, 1])
def test_between(codec):
    v = np.array([[1.0, 1.06, -3.3, 0.0, 200.0]])
    sc = np.ones(1, np.float32)
    q = oc.encode_nearest(v, codec)
    assert os_.between(q, sc, v, 0 * v, codec).all()
    up = oc.encode_nearest(v * 1.13, codec)
    up[0, 3] = 1
    assert not os_.between(up, sc, v, 0 * v, codec).any()
    border = np.array([[1.0625]])   # halfway between 1 and 1.125: either, given slack
    for c in (1.0, 1.125):
        assert os_.between(oc.encode_nearest(np.array([[c]]), codec), sc, border, np.array([[1e-9]]), codec).all()
