"""Gradients of confident routers, each to its own digits, against the gradient by differences (oracle/gate.py).

Tolerances, u = 2^-24, X the largest |logit| or distance from the row's maximum (at most 90: beyond, scores are below 2^-126
and covered by TINY): an exponential is within (3 X + 2) u, so a sigmoid's score and complement, one reciprocal (2 u) and two
operations more, within (3 X + 6) u; a score over the scores' sum within e = (6 X + 30) u.  A quotient's gradient
u_i (x_i - sum u x) has its terms' errors: x_i within 4 u (two products, a sum, a difference), the sum's terms within e + 4 u
and 22 u of additions.  With size the magnitudes of what remains after the terms of i itself cancel (at least a half of
u_i |x_i|, where no score is above a half), the whole is within 4 e + 60 u, the complement's (3 X + 6) u more: below
(40 X + 300) u size.  Values below the fp32 normal range may be flushed."""
import numpy as np
import pytest
import torch

import mxfp8_quantized_moe_amd as fm
from oracle import gate as og
from oracle.swiglu import round_bf16
from gpu_helpers import DEV, note, bf16_dev, i32_dev, host, bf16_bits_to_f64

pytestmark = pytest.mark.gpu

U, TINY = 2.0 ** -24, 2.0 ** -126


def dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def device_logits(z, dtype):
    """Device logits and their fp64 values."""
    if dtype == "bf16":
        bits = round_bf16(z)
        return bf16_dev(bits), bf16_bits_to_f64(bits)
    z32 = z.astype(np.float32)
    return dev(z32), z32.astype(np.float64)


def spread(z, sigmoid):
    e = og.eligible_logits(z)
    with np.errstate(invalid="ignore"):
        d = np.abs(e) if sigmoid else e.max(axis=1, keepdims=True) - e
    return float(np.minimum(d[e > -np.inf], 90.0).max())


def check(z, zd, ids, dw, dprob, sigmoid, renorm, offs, what, factor=(40, 300)):
    kw = dict(dprob=dev(dprob), dloss=dev(np.array([0.75], np.float32)), seq_offs=i32_dev(offs)) if dprob is not None else {}
    score = int(sigmoid)
    note("moe_gate_backward " + what)
    if dw is None:
        got = fm.moe_balance_loss_backward(zd, kw["dprob"], kw["dloss"], kw["seq_offs"], score)
    else:
        got = fm.moe_gate_backward(zd, i32_dev(ids), dev(dw), score, None, renorm, 2.0, **kw)
    dz, size = og.backward_by_differences(z, ids, dw, sigmoid, None, renorm, 2.0, dprob, 0.75, offs)
    bf16 = got.dtype == torch.bfloat16
    g = bf16_bits_to_f64(host(got)) if bf16 else host(got).astype(np.float64)
    most = max(0 if dw is None else 2 * np.abs(dw).max(), 0 if dprob is None else dprob.max())
    tol = (factor[0] * spread(z, sigmoid) + factor[1]) * U * size + (2.0 ** -8 * np.abs(dz) if bf16 else 0) + 8 * TINY * (1 + most)
    bad = np.abs(g - dz) - tol
    assert np.all(bad <= 0), f"{what}: {np.unravel_index(np.argmax(bad), bad.shape)} got {g.flat[np.argmax(bad)]} want {dz.flat[np.argmax(bad)]}"


@pytest.mark.parametrize("E,k", [(4, 1), (6, 2), (16, 1), (16, 4), (64, 6), (200, 8), (255, 8), (512, 4), (1024, 16)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_confident_sigmoid(E, k, dtype):
    """Half the experts at logits 8 .. 30, where 1 - s is e^-8 .. e^-30 of the score; the others around 0."""
    rng = np.random.default_rng(E * 3 + k)
    T = 40
    z = np.where(rng.random((T, E)) < 0.5, rng.uniform(8, 30, size=(T, E)), rng.standard_normal((T, E)))
    z[:, rng.permutation(E)[: max(k, 3)]] = rng.uniform(8, 30, size=(T, max(k, 3)))
    zd, z = device_logits(z, dtype)
    ids, _ = og.gate(z, k, True)
    dw = rng.standard_normal((T, k)).astype(np.float32)
    dprob = rng.random((2, E)).astype(np.float32)
    for renorm in (False, True):
        for a, b in ((dw, None), (None, dprob), (dw, dprob)):
            check(z, zd, ids, a, b, True, renorm, [13, 40], f"confident sigmoid {E} top {k} {dtype} renorm {renorm} {a is None} {b is None}")


def test_single_confident_expert():
    """Top 1 of a sigmoid router, logits 8 .. 30: the gradient is dw s (1 - s), never 0."""
    z = np.linspace(8, 30, 45)[:, None].repeat(2, 1)
    z[:, 1] = -1.0
    zd, z = device_logits(z, "f32")
    ids = np.zeros((45, 1), np.int32)
    check(z, zd, ids, np.ones((45, 1), np.float32), None, True, False, None, "one confident expert")
