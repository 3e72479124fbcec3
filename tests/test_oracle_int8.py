"""The integer oracle against pure-Python arithmetic, and mistakes it must notice."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import int8 as oi
from oracle.swiglu import round_bf16


def nearest_even(v: Fraction) -> int:
    lo = v.numerator // v.denominator
    d = v - lo
    return lo + (1 if d > Fraction(1, 2) or (d == Fraction(1, 2) and lo % 2) else 0)


def test_codes_by_fractions():
    rng = np.random.default_rng(1)
    x = round_bf16(np.concatenate([rng.standard_normal((6, 24)), np.zeros((1, 24)), 1e-30 * rng.standard_normal((1, 24))]))
    q, s = oi.quantize_rowwise(x)
    f = oi.bf16_to_f32(x)
    for r in range(len(x)):
        amax = max(abs(float(v)) for v in f[r])
        exact = Fraction(127) / Fraction(max(amax, float(np.float32(1e-12))))
        assert abs(Fraction(float(s[r])) - exact) <= 2 * exact / 2 ** 24 + exact / 2 ** 47   # two roundings
        for c in range(24):
            y = np.float32(f[r, c] * s[r])                     # one rounded product
            assert q[r, c] == nearest_even(Fraction(float(np.clip(y, -127, 127))))
    assert not q[6].any() and s[6] == np.float32(127) * (np.float32(1) / np.float32(1e-12))
    assert (np.abs(q[:6].astype(int)).max(axis=1) == 127).all()   # the row's largest value is the largest code


def test_scale_is_torchs():
    torch = pytest.importorskip("torch")
    x = round_bf16(np.random.default_rng(3).standard_normal((2000, 8)))
    t = torch.from_numpy(oi.bf16_to_f32(x))
    assert (oi.quantize_rowwise(x)[1] == (127.0 / t.abs().amax(1)).numpy()).all()


def test_ties_go_to_even():
    x = round_bf16(np.array([[127, 0.5, 1.5, 2.5, -0.5, -1.5, -2.5, 126.5]]))
    q, s = oi.quantize_rowwise(x)
    assert s[0] == 1.0
    assert q[0].tolist() == [127, 0, 2, 2, 0, -2, -2, 126]


@pytest.mark.parametrize("offs", [[3, 3, 7], [5, 2, 9], [-1, 4, 100]])
def test_product_by_loops(offs):
    rng = np.random.default_rng(2)
    M, N, K, E = 8, 5, 16, 3
    a, b = rng.integers(-128, 128, (M, K)).astype(np.int8), rng.integers(-128, 128, (E, N, K)).astype(np.int8)
    sa, sb = rng.uniform(1, 3, M).astype(np.float32), rng.uniform(1, 3, (E, N)).astype(np.float32)
    got = oi.mm_grouped_m(a, sa, b, sb, np.array(offs, np.int32))
    hi, group = 0, [-1] * M
    for e, o in enumerate(offs):
        new = max(hi, min(max(o, 0), M))
        for m in range(hi, new):
            group[m] = e
        hi = new
    for m in range(M):
        for n in range(N):
            if group[m] < 0:
                assert np.isnan(got[m, n])
                continue
            acc = sum(int(a[m, k]) * int(b[group[m], n, k]) for k in range(K))
            assert got[m, n] == pytest.approx(acc / (float(sa[m]) * float(sb[group[m], n])), rel=1e-15)
    wrong = oi.mm_grouped_m(a, sa, b, sb[:, ::-1], np.array(offs, np.int32))   # a planted mistake: another channel's scale
    rows = [m for m in range(M) if group[m] >= 0]
    assert not np.allclose(got[rows], wrong[rows])
