"""The few-token oracle against loops, and its bound against mistakes it has to notice."""
import math

import numpy as np
import pytest

from oracle import few as of
from oracle.quant import bf16_to_f32
from oracle.swiglu import round_bf16


def data(T=4, K=8, F=6, E=3, k=2, seed=0):
    rng = np.random.default_rng(seed)
    bf = lambda v: bf16_to_f32(round_bf16(v)).astype(np.float64)
    ids = rng.integers(-1, E, (T, k))
    ids[0] = 1                                   # an expert named twice
    ids[1] = -1                                  # a token without an expert
    return bf(rng.standard_normal((T, K))), ids, rng.random((T, k)), bf(rng.standard_normal((E, 2 * F, K))), \
        bf(rng.standard_normal((E, K, F)))


@pytest.mark.parametrize("seed", [0, 1])
def test_by_loops(seed):
    x, ids, w, w1, w2 = data(seed=seed)
    y, bound = of.block(x, ids, w, w1, w2)
    T, K = x.shape
    F = w1.shape[1] // 2
    for t in range(T):
        want = [0.0] * K
        for j, e in enumerate(ids[t]):
            if e < 0:
                continue
            a = []
            for f in range(F):
                g = sum(x[t, i] * w1[e, f, i] for i in range(K))
                u = sum(x[t, i] * w1[e, F + f, i] for i in range(K))
                a.append(float(bf16_to_f32(round_bf16(np.array([g / (1 + math.exp(-g)) * u])))[0]))
            for c in range(K):
                want[c] += w[t, j] * sum(a[f] * w2[e, c, f] for f in range(F))
        assert y[t] == pytest.approx(want, rel=1e-12, abs=1e-12)
    assert (y[1] == 0).all() and (bound[1] < 1e-37).all()


def test_bound_notices():
    x, ids, w, w1, w2 = data(T=8, K=64, F=48, seed=3)
    y, bound = of.block(x, ids, w, w1, w2)
    F = w1.shape[1] // 2
    wrong = [of.block(x, ids, w[:, ::-1], w1, w2)[0],                                    # another slot's weight
             of.block(x, ids, w, np.concatenate([w1[:, F:], w1[:, :F]], 1), w2)[0],      # gate and up exchanged
             of.block(x, np.where(ids >= 0, (ids + 1) % 3, ids), w, w1, w2)[0],          # another expert
             of.block(np.where(np.arange(64) < 63, x, 0), ids, w, w1, w2)[0]]            # the last input left out
    for v in wrong:
        assert (np.abs(v - y) > bound).mean() > 0.3
    # plain fp32 in another order stays inside
    x32, a1, a2 = x.astype(np.float32), w1.astype(np.float32), w2.astype(np.float32)
    got = np.zeros_like(y)
    for t in range(len(x)):
        for j, e in enumerate(ids[t]):
            if e >= 0:
                h = (a1[e][:, ::-1] @ x32[t, ::-1]).astype(np.float32)
                a = bf16_to_f32(round_bf16((of.silu(h[:F].astype(np.float64)) * h[F:])))
                got[t] += w[t, j] * (a2[e] @ a).astype(np.float64)
    got = bf16_to_f32(round_bf16(got))
    assert (np.abs(got - y) <= bound).all()
