"""The kept SwiGLU at gates between -104 and -87, whose sigmoid lies below 2^-126 but not below fp32's spacing: the
activation and both gradients keep the digits that such a sigmoid has."""
import numpy as np
import pytest

import mxfp8_quantized_moe_amd as fm
from oracle import quant as oq
from oracle import saved as os_
from oracle.quant import bf16_to_f32
from oracle.swiglu import round_bf16
from gpu_helpers import note, bf16_dev, u8_dev, host, bf16_bits_to_f64

pytestmark = pytest.mark.gpu

TINY = 2.0 ** -149   # fp32's spacing below 2^-126


def far_rows(R, F, gates):
    """Rows of near gates, of far ones, and of both; ups as large as bf16 lets a product with them be a normal number."""
    rng = np.random.default_rng(R + F)
    h = rng.standard_normal((R, 2 * F))
    for r in range(R):
        if r % 3:
            cols = np.arange(F) if r % 3 == 1 else rng.permutation(F)[:F // 2]
            h[r, cols] = rng.permutation(np.resize(gates, cols.size))
            h[r, F + cols] *= (1e4, 1e25, 1e36)[r // 3 % 3]
    return round_bf16(h)


def near(got, v, slack, what):
    """As bf16: half a step of the value, 2^-8 of it at most, or of bf16's spacing 2^-133 below 2^-126; infinity beyond
    the range of fp32 (gate 300 with an up of 1e36 times a normal number)."""
    got = bf16_bits_to_f64(got)
    over = np.abs(v) - slack >= 2.0 ** 128
    assert (got[over] == np.copysign(np.inf, v[over])).all(), what
    off = np.abs(np.where(over, 0, got) - np.where(over, 0, v)) - (slack + np.maximum(2.0 ** -8 * (np.abs(v) + slack), 2.0 ** -134))
    assert (off <= 0).all(), f"{what}: worst {off.max()} at {np.argwhere(off > 0)[0]}"


@pytest.mark.parametrize("codec", [0, 1])
@pytest.mark.parametrize("R,F", [(11, 96), (10, 1056), (2049, 160), (9, 16416)])
def test_forward(R, F, codec):
    note(f"swiglu_quantize_rowwise_save far gates {R}x{F} codec {codec}")
    h = far_rows(R, F, np.concatenate([np.arange(-104, -80, 0.5), np.arange(80, 104, 0.5), [-np.finfo(np.float32).max / 2, 300]]))
    a2, q, s, _, _ = fm.swiglu_quantize_rowwise_save(bf16_dev(h), codec=codec, keep_bf16=True)
    v = bf16_to_f32(h).astype(np.float64)
    with np.errstate(over="ignore"):
        a = os_.forward(v)
    g, u = np.abs(v[:, :F]), np.abs(v[:, F:])
    # ten half steps as elsewhere; a sigmoid below 2^-126 is off by its spacing at most (the exponential's rounding and the
    # product with the reciprocal), and so is its product with the gate
    far = v[:, :F] < -87
    slack = 10 * 2.0 ** -24 * np.abs(a) + np.where(far, u * (g + 1) * TINY, 0) + 2.0 ** -150
    near(host(a2), a, slack, "a2")
    assert (bf16_bits_to_f64(host(a2))[(v[:, :F] < -87) & (v[:, :F] > -103) & (u > 1e3)] != 0).all()
    held = (np.abs(a) < 2.0 ** 127).all(1)            # a row with an infinity has no scale
    assert os_.between(host(q), host(s), a, slack, codec)[held].all()


@pytest.mark.parametrize("codec", [0, 1])
@pytest.mark.parametrize("R,F", [(11, 96), (10, 1056), (2049, 160), (9, 16416)])
def test_backward(R, F, codec):
    note(f"swiglu_backward_quantize_rowwise_saved far gates {R}x{F} codec {codec}")
    hq, hs = oq.quantize_mx_lastdim(far_rows(R, F, np.array([-104, -96, -88, -80, 80, 88, 96, 104, -72, -56, 56])), 1)
    d = round_bf16(np.random.default_rng(F).standard_normal((R, F)))
    dh1, q, s, a2 = fm.swiglu_backward_quantize_rowwise_saved(bf16_dev(d), u8_dev(hq), u8_dev(hs), codec=codec, want_a2=True)
    v, df = os_.kept_values(hq, hs), bf16_bits_to_f64(d)
    assert {-96, -88} <= set(np.unique(v[:, :F]))
    dh, slack = os_.backward(df, v)
    g, u = np.abs(v[:, :F]), np.abs(v[:, F:])
    far = v[:, :F] < -87
    slack += np.concatenate([np.where(far, (np.abs(df) * u + 1) * (g + 1) * TINY, 0), np.where(far, np.abs(df) * (g + 1) * TINY, 0)], 1)
    near(host(dh1), dh, slack, "dh1")
    a = os_.forward(v)
    near(host(a2), a, 10 * 2.0 ** -24 * np.abs(a) + np.where(far, u * (g + 1) * TINY, 0) + 2.0 ** -150, "a2")
    assert (bf16_bits_to_f64(host(a2))[far & (g < 100) & (u > 1e3)] != 0).all()
    assert os_.between(host(q), host(s), dh, slack, codec).all()
