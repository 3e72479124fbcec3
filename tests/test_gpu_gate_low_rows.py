"""The balance loss of sigmoid rows whose scores lie below the fp32 range: each token still counts one share in all, and its
gradient is that of the shares, down to scores that are 0 in 64 bits (a row of the lowest value), which have none.  Tolerances as in test_gpu_gate.py (loss: (6 X + 70) u) and test_gpu_gate_confident.py."""
import numpy as np
import pytest
import torch

import mxfp8_quantized_moe_amd as fm
from oracle import gate as og
from oracle.swiglu import round_bf16
from gpu_helpers import DEV, note, host, bf16_dev, i32_dev, bf16_bits_to_f64

pytestmark = pytest.mark.gpu

U, TINY = 2.0 ** -24, 2.0 ** -126
LOWEST = float(np.finfo(np.float32).min)


def dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def rows(rng, T, E, kind):
    z = rng.uniform(0, 3, size=(T, E))
    if kind == "mixed":                                  # a level of its own for each row, some of them ordinary
        return z + rng.choice([0.0, -1.0, -5.0, -86.0, -88.0, -95.0, -400.0], size=(T, 1))
    if kind == "lowest":
        z = np.full((T, E), LOWEST)
        z[::2, ::3] = -np.inf
        z[5] = -np.inf
        return z
    return z + kind


@pytest.mark.parametrize("T,E,k", [(40, 9, 2), (70, 16, 1), (33, 64, 6), (50, 100, 3), (17, 255, 8), (20, 256, 8), (9, 400, 4),
                                   (12, 1000, 10)])
@pytest.mark.parametrize("kind", [-3.0, -84.0, -90.0, -100.0, -1000.0, "mixed", "lowest"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_low_rows(T, E, k, kind, dtype):
    what = f"low rows {T}x{E} top {k} {kind} {dtype}"
    note(what)
    rng = np.random.default_rng(T + E)
    z = rows(rng, T, E, kind)
    if dtype == "bf16":
        bits = round_bf16(np.where(np.isfinite(z), np.maximum(z, -3.38e38), 0))
        bits[np.isneginf(z)] = 0xFF80
        zd, z = bf16_dev(bits), (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    else:
        zd, z = dev(z.astype(np.float32)), z.astype(np.float32).astype(np.float64)
    offs, coef = [T // 3, T - 2], 0.4
    mask = rng.random(T) < 0.8
    ids, w, loss, counts, dprob = fm.moe_gate_balance(zd, k, coef, i32_dev(offs), fm.GATE_SIGMOID, token_mask=dev(mask))
    h = host(ids)
    np.testing.assert_array_equal(h, og.gate(z, k, True, None, mask)[0])
    p = og.loss_shares(z, True)
    assert np.array_equal(p.any(axis=1), (z > -709).any(axis=1))
    want, seq = 0.0, [(0, offs[0]), (offs[0], offs[1])]
    for s, (lo, hi) in enumerate(seq):
        t = np.arange(lo, hi)[mask[lo:hi]]
        c = np.bincount(h[t][h[t] >= 0], minlength=E)
        np.testing.assert_array_equal(host(counts)[s], c)
        want += coef / 2 * (c * E / (k * len(t)) * p[t].mean(axis=0)).sum()
    X = 90.0
    assert abs(float(loss) - want) <= (6 * X + 70) * U * want, f"{what}: {float(loss)} want {want}"
    again = fm.moe_balance_loss(zd, ids, coef, i32_dev(offs), fm.GATE_SIGMOID, dev(mask))
    assert abs(float(again[0]) - want) <= (6 * X + 70) * U * want and torch.equal(again[1], counts)
    d = host(dprob)
    dl = np.array([3.0], np.float32)
    got = fm.moe_balance_loss_backward(zd, dprob, dev(dl), i32_dev(offs), fm.GATE_SIGMOID, dev(mask))
    dz, size = og.backward_by_differences(z, h, None, True, mask, False, 1.0, d, 3.0, offs)
    g = bf16_bits_to_f64(host(got)) if dtype == "bf16" else host(got).astype(np.float64)
    tol = (40 * X + 300) * U * size + (2.0 ** -8 * np.abs(dz) if dtype == "bf16" else 0) + 8 * TINY * (1 + 3 * d.max())
    assert np.all(np.abs(g - dz) <= tol), what
    assert np.all(g[~mask] == 0)
