"""GPU parity of the router gate, the balance loss and their backward against the fp64 oracle (oracle/gate.py).

ids and counts are whole numbers and must match exactly.  Tolerances, with u = 2^-24 and X the largest distance
|logit - row maximum| (softmax) or |logit| (sigmoid) of a case: an exponential of x costs its argument's rounding
(u |x|), the product with log2 e (constant and product: 2 u |x|) and 2 u of its own, so (3 X + 2) u relative; the
denominator holds the same error, at most 22 additions and a reciprocal (2 u); the product one more.  A score is
within (6 X + 30) u relative, its renormalisation twice that; values below the fp32 normal range may be flushed
(2^-126 absolute).  The loss adds fp32 sums
over at most 32 tokens of a lane, then over the lanes' groups four at a time: at most 35 roundings.  A logit's gradient
is a sum of terms of total magnitude `size` (oracle), each a product of at most four such factors: (24 X + 160) u size.
"""
import numpy as np
import pytest
import torch

import mxfp8_quantized_moe_amd as fm
from oracle import gate as og
from oracle import route as rt
from oracle.swiglu import round_bf16
from gpu_helpers import DEV, note, bf16_dev, i32_dev, host, bf16_bits_to_f64

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TINY = 2.0 ** -126


def dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def make_logits(rng, T, E, dtype, dead=False, sigma=2.0, pad=0):
    """(device logits, a slice of rows pad wider whose tail is +inf, and their fp64 values)."""
    z = rng.standard_normal((T, E)) * sigma
    if dead and T:
        z[rng.random((T, E)) < 0.25] = -np.inf
        z[rng.random((T, E)) < 0.02] = np.nan
        z[rng.random(T) < 0.1] = -np.inf
        z[0] = -np.inf
        z[T // 2, : E // 2] = np.finfo(np.float32).min      # the lowest finite value: still eligible
        z[T - 1, E - 1] = np.inf
    wide = np.full((T, E + pad), np.inf)
    wide[:, :E] = z
    if dtype == "bf16":
        fin = np.where(np.isfinite(wide), np.clip(wide, -3.38e38, 3.38e38), 0)
        bits = round_bf16(fin)
        bits[np.isneginf(wide)], bits[np.isposinf(wide)], bits[np.isnan(wide)] = 0xFF80, 0x7F80, 0x7FC0
        return bf16_dev(bits)[:, :E], (bits[:, :E].astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    w32 = wide.astype(np.float32)
    return dev(w32)[:, :E], w32[:, :E].astype(np.float64)


def spread(z, sigmoid):
    """X of the tolerances; scores further down than 2^-126 are covered by TINY."""
    e = og.eligible_logits(z)
    fin = e > -np.inf
    if not fin.any():
        return 0.0
    if sigmoid:
        d = np.abs(e[fin])
    else:
        with np.errstate(invalid="ignore"):
            d = (e.max(axis=1, keepdims=True) - e)[fin]
    return float(np.minimum(d, 90.0).max())


def check_gate(got, z, topk, sigmoid, bias, mask, renorm, scale, what):
    ids, w = og.gate(z, topk, sigmoid, bias, mask, renorm, scale)
    np.testing.assert_array_equal(host(got[0]), ids, err_msg=what)
    tol = (6 * spread(z, sigmoid) + 30) * U * (2 if renorm else 1)
    err = np.abs(host(got[1]) - w)
    assert np.all(err <= tol * np.abs(w) + 4 * TINY * scale), f"{what}: {np.max(err)}"
    return ids


def check_loss(got, z, ids, coef, offs, sigmoid, mask, what):
    loss, counts, dprob = og.balance(z, ids, coef, offs, sigmoid, mask)
    np.testing.assert_array_equal(host(got[1]), counts, err_msg=what)
    assert np.all(np.abs(host(got[2]) - dprob) <= 2 * U * dprob), f"{what} dprob"
    assert abs(host(got[0])[0] - loss) <= (6 * spread(z, sigmoid) + 70) * U * abs(loss) + TINY, f"{what} loss"
    return dprob


# tokens, experts, topk
SHAPES = [(1, 1, 1), (1, 16, 1), (3, 2, 2), (5, 7, 7), (33, 16, 1), (64, 64, 6), (17, 63, 5), (129, 65, 8), (40, 128, 4),
          (31, 200, 12), (50, 256, 8), (9, 257, 3), (21, 512, 10), (7, 777, 64), (12, 1024, 16), (700, 60, 4), (3000, 8, 2),
          (9, 64, 64), (5, 200, 40), (6, 16, 16), (4, 300, 17)]


@pytest.mark.parametrize("T,E,k", SHAPES)
@pytest.mark.parametrize("sigmoid", [False, True])
def test_gate(T, E, k, sigmoid):
    rng = np.random.default_rng(T * 1009 + E * 7 + k + sigmoid)
    for dtype in ("f32", "bf16"):
        dead = (T + E) % 2 == 0
        zd, z = make_logits(rng, T, E, dtype, dead, pad=(T + k) % 3)
        mask = rng.random(T) < 0.8 if T % 2 else None
        bias = (0.2 * rng.standard_normal(E)).astype(np.float32) if (E + k) % 3 == 0 else None
        renorm, scale = bool((T + k) % 2), 2.5 if E % 2 else 1.0
        what = f"{T}x{E} top {k} {dtype} sigmoid {sigmoid} dead {dead} mask {mask is not None} bias {bias is not None}"
        note("moe_gate " + what)
        got = fm.moe_gate(zd, k, fm.GATE_SIGMOID if sigmoid else fm.GATE_SOFTMAX, dev(bias),
                          dev(None if mask is None else mask.astype(np.uint8)), renorm, scale)
        check_gate(got, z, k, sigmoid, bias, mask, renorm, scale, what)


def test_ties_go_to_the_lower_index():
    note("moe_gate ties")
    z = np.zeros((70, 100), np.float32)
    z[:, 40:60] = 1.0
    z[::2, 3] = 1.0
    z[1::2, 99] = -0.0                                      # -0 equals +0
    for sigmoid in (fm.GATE_SOFTMAX, fm.GATE_SIGMOID):
        for bias in (None, np.zeros(100, np.float32)):
            ids, w = fm.moe_gate(dev(z), 25, sigmoid, dev(bias))
            want = og.gate(z.astype(np.float64), 25, bool(sigmoid), bias)[0]
            np.testing.assert_array_equal(host(ids), want)
    want = og.gate(np.zeros((2, 1000)), 64, False)[0]
    np.testing.assert_array_equal(host(fm.moe_gate(torch.zeros(2, 1000, device=DEV), 64)[0]), want)


def test_bias_decides_in_64_bits():
    """Keys that fp32 cannot tell apart: score + bias differ by less than an fp32 step of the key."""
    note("moe_gate close keys")
    rng = np.random.default_rng(5)
    T, E, k = 500, 64, 4
    z = (rng.standard_normal((T, 1)) + 1e-6 * rng.integers(0, 8, size=(T, E))).astype(np.float32)
    for b0 in (0.0, 1.0, -3.0):
        bias = np.full(E, b0, np.float32)
        for sigmoid in (False, True):
            got = fm.moe_gate(dev(z), k, int(sigmoid), dev(bias))
            np.testing.assert_array_equal(host(got[0]), og.gate(z.astype(np.float64), k, sigmoid, bias)[0])


def test_order_below_the_truncated_keys():
    """Logits that differ in their last four bits only, and ties of them."""
    note("moe_gate last bits")
    rng = np.random.default_rng(15)
    for E, k in ((16, 3), (64, 8), (256, 8), (200, 12), (1000, 20)):
        z = (rng.choice([1.0, -1.0, 3.0], size=(200, 1)) * (1 + rng.integers(0, 16, size=(200, E)) * 2.0 ** -23)).astype(np.float32)
        z[::3, E // 2:] = -5.0
        got = fm.moe_gate(dev(z), k)
        np.testing.assert_array_equal(host(got[0]), og.gate(z.astype(np.float64), k, False)[0])


def test_one_lane_gives_all_choices():
    """All of a row's largest logits in one lane (experts 4 l + 0..3 of each chunk of 64, of 256 beyond 256 experts): more
    than eight, so that what the lane keeps runs out."""
    note("moe_gate one lane")
    rng = np.random.default_rng(16)
    for E, step in ((256, 64), (1024, 256), (128, 64)):
        mine = [e for e in range(E) if (e % step) // 4 == 5]
        z = rng.standard_normal((40, E)).astype(np.float32)
        z[:, mine] = 10 + rng.standard_normal((40, len(mine))).astype(np.float32)
        z[::2, mine] = np.float32(10) + np.float32(2.0 ** -20) * rng.integers(0, 16, size=(20, len(mine)))
        for bias in (None, np.zeros(E, np.float32)):
            for k in (7, 8, 9, 16):
                got = fm.moe_gate(dev(z), k, fm.GATE_SIGMOID, dev(bias))
                np.testing.assert_array_equal(host(got[0]), og.gate(z.astype(np.float64), k, True, bias)[0])


def test_nan_patterns():
    """Quiet and signalling NaN of either sign, and -inf, are no expert; +inf comes first."""
    note("moe_gate NaN patterns")
    z = np.random.default_rng(17).standard_normal((8, 32)).astype(np.float32)
    bits = z.view(np.uint32).copy()
    for e, b in ((0, 0x7FC00000), (3, 0x7F800001), (9, 0xFFC00000), (17, 0xFF800001), (30, 0x7FFFFFFF), (31, 0xFF800000)):
        bits[:, e] = b
    bits[4:, 12] = 0x7F800000
    zd, z = torch.from_numpy(bits.view(np.int32)).to(DEV).view(torch.float32), bits.view(np.float32)
    half = torch.from_numpy((bits >> 16).astype(np.uint16).view(np.int16)).to(DEV).view(torch.bfloat16)
    zh = ((bits >> 16) << 16).view(np.float32)   # 0x7F800001 is +inf and 0xFF800001 -inf in bf16; 0x7FFF is a NaN
    for t, v in ((zd, z), (half, zh)):
        for sigmoid in (False, True):
            for bias in (None, np.full(32, 0.25, np.float32)):
                ids, w = fm.moe_gate(t, 32, int(sigmoid), dev(bias))
                with np.errstate(invalid="ignore"):   # a signalling NaN, widened
                    want, ww = og.gate(v.astype(np.float64), 32, sigmoid, bias)
                np.testing.assert_array_equal(host(ids), want)
                assert np.all(np.abs(host(w) - ww) <= 1e-5 * ww + 4 * TINY)


def test_infinite_bias():
    note("moe_gate infinite bias")
    z = np.random.default_rng(6).standard_normal((9, 12)).astype(np.float32)
    bias = np.zeros(12, np.float32)
    bias[[2, 5]], bias[7], bias[0] = np.inf, -np.inf, np.nan
    ids = host(fm.moe_gate(dev(z), 12, fm.GATE_SIGMOID, dev(bias))[0])
    assert np.all(ids[:, :2] == [2, 5]) and np.all(ids[:, 10:] == -1) and not np.any((ids == 7) | (ids == 0))


def test_largest_keys():
    """Infinite biases go before the largest finite one, which swallows the scores: each kind's ties to the lower index,
    chosen or left out."""
    note("moe_gate largest keys")
    big = np.finfo(np.float32).max
    z = np.random.default_rng(8).standard_normal((70, 40)).astype(np.float32)
    z[1, :] = -np.inf
    z[2, ::2] = np.nan
    z[3, 5], z[3, 30] = np.inf, -big
    bias = np.zeros(40, np.float32)
    bias[[5, 21, 39]], bias[[2, 20, 30]], bias[11], bias[12], bias[13] = np.inf, big, -big, -0.0, -np.inf
    for sigmoid in (0, 1):
        for k in (1, 2, 3, 5, 6, 7, 40):
            ids, w = fm.moe_gate(dev(z), k, sigmoid, dev(bias))
            want, _ = og.gate(z.astype(np.float64), k, bool(sigmoid), bias)
            np.testing.assert_array_equal(host(ids), want)


# tokens, experts, topk, sequence ends (None: no offsets)
LOSSES = [(1, 4, 1, None), (0, 8, 2, None), (0, 8, 2, [0, 0]), (64, 16, 1, [64]), (100, 16, 1, [10, 10, 50, 90]),
          (333, 64, 6, [1, 2, 3, 333]), (50, 256, 8, [20, 5, 70, 50]), (2000, 30, 3, None), (40, 1000, 5, [0, 40]),
          (600, 9, 2, list(range(5, 605, 6))), (5000, 64, 6, [1234, 4999]), (130, 3, 1, [-5, 0, 130]),
          (20, 513, 4, [300, 400])]


@pytest.mark.parametrize("case", range(len(LOSSES)))
@pytest.mark.parametrize("sigmoid", [False, True])
def test_balance_loss(case, sigmoid):
    T, E, k, offs = LOSSES[case]
    rng = np.random.default_rng(case * 2 + sigmoid)
    score = int(sigmoid)
    for dtype in ("f32", "bf16"):
        zd, z = make_logits(rng, T, E, dtype, dead=case % 2 == 1, pad=case % 2)
        mask = rng.random(T) < 0.7 if case % 3 == 1 else None
        md = dev(mask)                                       # torch.bool
        od = None if offs is None else i32_dev(offs)
        what = f"{T}x{E} top {k} ends {offs and offs[:6]} {dtype} sigmoid {sigmoid}"
        note("moe_balance_loss " + what)
        ids, w, *rest = fm.moe_gate_balance(zd, k, 0.3, od, score, token_mask=md)
        ref = check_gate((ids, w), z, k, sigmoid, None, mask, False, 1.0, what)
        check_loss(rest, z, ref, 0.3, offs, sigmoid, mask, what)
        plain = fm.moe_gate(zd, k, score, token_mask=md)
        assert torch.equal(plain[0], ids) and torch.equal(plain[1], w)
        # choices made elsewhere: repeated, dropped and out-of-range ids
        other = rng.integers(-1, E + 1, size=(T, k)).astype(np.int32)
        got = fm.moe_balance_loss(zd, i32_dev(other), -2.0, od, score, md)
        loss, counts, dprob = og.balance(z, other, -2.0, offs, sigmoid, mask)
        np.testing.assert_array_equal(host(got[1]), counts)
        assert np.all(np.abs(host(got[2]) - dprob) <= 2 * U * np.abs(dprob))
        assert abs(host(got[0])[0] - loss) <= (6 * spread(z, sigmoid) + 70) * U * abs(loss) + TINY


@pytest.mark.parametrize("S,E,n", [(64, 256, 2), (400, 1024, 1), (3, 1024, 50), (65535, 16, 1)])
def test_loss_of_collapsed_routing(S, E, n):
    """Every token on one expert: a sequence adds E f P = E, the most there is, S times over.  The sum over sequences
    and slices of experts rounds each by 2^-54, far below the tolerance."""
    note(f"moe_gate_balance collapsed {S} sequences of {n} x {E}")
    z = np.zeros((S * n, E))
    z[:, 3] = 40.0
    offs = [n * (s + 1) for s in range(S)]
    zd = dev(z.astype(np.float32))
    for sigmoid in (0, 1):
        ids, w, *rest = fm.moe_gate_balance(zd, 1, 0.5, i32_dev(offs), sigmoid)
        assert bool((ids == 3).all())
        loss, counts, dprob = og.balance(z, host(ids), 0.5, offs, bool(sigmoid))
        if not sigmoid:
            assert abs(loss - 0.5 * E) < 1e-9 * E
        np.testing.assert_array_equal(host(rest[1]), counts)
        assert np.all(np.abs(host(rest[2]) - dprob) <= 2 * U * np.abs(dprob))
        assert abs(host(rest[0])[0] - loss) <= (6 * spread(z, bool(sigmoid)) + 70) * U * abs(loss) + TINY


def test_counts_agree_with_the_routing():
    rng = np.random.default_rng(12)
    zd, z = make_logits(rng, 1000, 64, "f32")
    note("counts against moe_route")
    ids, _, _, counts, _ = fm.moe_gate_balance(zd, 6, 0.01)
    assert torch.equal(counts[0], fm.moe_route(ids, 64)[0])


BACK = [(1, 1, 1, None), (3, 2, 2, [3]), (33, 16, 1, [10, 33]), (64, 64, 6, None), (129, 65, 8, [0, 64, 100]),
        (31, 200, 12, [31]), (50, 256, 8, [7, 50]), (9, 777, 64, None), (12, 1024, 16, [5]), (700, 60, 4, [100, 350, 700]),
        (300, 10, 3, list(range(3, 303, 4)))]


@pytest.mark.parametrize("case", range(len(BACK)))
@pytest.mark.parametrize("sigmoid", [False, True])
def test_backward(case, sigmoid):
    T, E, k, offs = BACK[case]
    rng = np.random.default_rng(case * 2 + sigmoid)
    score = int(sigmoid)
    for dtype, renorm in (("f32", False), ("f32", True), ("bf16", case % 2 == 0)):
        zd, z = make_logits(rng, T, E, dtype, dead=case % 2 == 0, pad=case % 2, sigma=1.5)
        mask = rng.random(T) < 0.7 if case % 3 == 1 else None
        md = dev(mask)
        od = None if offs is None else i32_dev(offs)
        ids, _ = og.gate(z, k, sigmoid, None, mask)
        if case % 4 == 3 and k > 2:
            ids[0, :3] = [ids[0, 0], ids[0, 0], -1]          # a repeated and a dropped choice
            ids[T - 1, 0] = E + 5                            # out of range
        dw = (1e-2 * rng.standard_normal((T, k))).astype(np.float32)
        dprob = (1e-3 * rng.random((1 if offs is None else len(offs), E))).astype(np.float32)
        dloss = np.array([0.75], np.float32)
        X = spread(z, sigmoid)
        for part in ("gate", "loss", "both"):
            what = f"{part} {T}x{E} top {k} {dtype} sigmoid {sigmoid} renorm {renorm}"
            note("moe_gate_backward " + what)
            kw = dict(dprob=dev(dprob), dloss=dev(dloss), seq_offs=od) if part != "gate" else {}
            if part == "loss":
                got = fm.moe_balance_loss_backward(zd, kw["dprob"], kw["dloss"], od, score, md)
            else:
                # flat, as moe_combine_backward gives it
                got = fm.moe_gate_backward(zd, i32_dev(ids), dev(dw).view(-1), score, md, renorm, 2.0, **kw)
            dz, size = og.backward(z, ids, None if part == "loss" else dw, sigmoid, mask, renorm, 2.0,
                                   None if part == "gate" else dprob.astype(np.float64), 0.75, offs)
            g = bf16_bits_to_f64(host(got)) if dtype == "bf16" else host(got).astype(np.float64)
            tol = (24 * X + 160) * U * size + (2.0 ** -8 * np.abs(dz) if dtype == "bf16" else 0) + 1e-33
            assert np.all(np.abs(g - dz) <= tol), f"{what}: {np.max(np.abs(g - dz) - tol)}"
            if mask is not None:
                assert np.all(g[~mask] == 0)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("odd", ["logits", "bias", "dprob", "dlogits"])
def test_arrays_one_element_off(dtype, odd):
    """Each array starting one element past an aligned place, 256 experts: what aligned copies give (ids equal, sums of
    another order within the tolerances' roundings), and nothing is written beside the outputs."""
    note(f"moe_gate {odd} one element off {dtype}")

    def place(name, t):
        if name != odd:
            return t
        flat = torch.full((t.numel() + 9,), 7.0, dtype=t.dtype, device=DEV)
        flat[1:1 + t.numel()] = t.view(-1)
        return flat[1:1 + t.numel()].view(t.shape)

    g = torch.Generator(device=DEV).manual_seed(11)
    T, E, k = 37, 256, 8
    z = torch.randn(T, E, generator=g, device=DEV).to(dtype)
    bias = 0.1 * torch.randn(E, generator=g, device=DEV)
    dw = torch.randn(T, k, generator=g, device=DEV)
    ids, w, loss, counts, dprob = fm.moe_gate_balance(z, k, 0.1, None, 1, bias, renormalize=True)
    got = fm.moe_gate_balance(place("logits", z), k, 0.1, None, 1, place("bias", bias), renormalize=True)
    assert torch.equal(got[0], ids) and torch.equal(got[3], counts) and torch.equal(got[4], dprob)
    assert bool(((got[1] - w).abs() <= 16 * U * w.abs()).all())       # eight positive scores summed, one division
    assert bool(((got[2] - loss).abs() <= 300 * U * loss).all())      # 256 positive scores, then the units' sums
    want = fm.moe_gate_backward(z, ids, dw, 1, renormalize=True, dprob=dprob)
    out = place("dlogits", torch.zeros(T, E, dtype=dtype, device=DEV))
    back = fm.moe_gate_backward(place("logits", z), ids, dw, 1, renormalize=True, dprob=place("dprob", dprob), dlogits=out)
    assert back is out
    # sums of at most 256 terms of the size of dw (at most 5) over the chosen scores (at least 8 / 2): both rounded
    size = 300 * U * 5 + (2.0 ** -7 * want.float().abs() if dtype == torch.bfloat16 else 0)
    assert bool(((back.float() - want.float()).abs() <= size).all())
    if odd == "dlogits":
        whole = out.as_strided((T * E + 9,), (1,), out.storage_offset() - 1)
        assert float(whole[0]) == 7.0 and bool((whole[T * E + 1:] == 7.0).all())


def test_masked_tokens_stay_zero():
    """An overflowed loss gradient and NaN weights' gradients do not reach masked or uncounted tokens."""
    note("moe_gate_backward masked")
    z = torch.randn(100, 24, device=DEV)
    mask = torch.arange(100, device=DEV) % 3 != 0
    ids, _, _, _, dprob = fm.moe_gate_balance(z, 4, 0.1, i32_dev([60]), token_mask=mask)
    dw = torch.randn(100, 4, device=DEV)
    dw[~mask] = float("nan")
    for bad in (float("inf"), float("nan")):
        for score in (0, 1):
            dz = fm.moe_gate_backward(z, ids, dw, score, mask, dprob=dprob, dloss=torch.full((1,), bad, device=DEV),
                                      seq_offs=i32_dev([60]))
            assert torch.count_nonzero(dz[~mask]) == 0
            assert torch.isfinite(dz[60:]).all()


def test_single_renormalised_choice_passes_nothing():
    note("moe_gate_backward single choice")
    z = torch.randn(300, 40, device=DEV)
    for score in (0, 1):
        ids, w = fm.moe_gate(z, 1, score, renormalize=True)
        assert torch.equal(w, torch.ones_like(w))
        dz = fm.moe_gate_backward(z, ids, torch.randn(300, 1, device=DEV), score, renormalize=True)
        assert torch.count_nonzero(dz) == 0


def test_outputs_given_and_refused():
    note("moe_gate outputs")
    z = torch.randn(30, 12, device=DEV)
    ids, w = torch.full((30, 3), 9, dtype=torch.int32, device=DEV), torch.empty(30, 3, device=DEV)
    a = fm.moe_gate(z, 3, ids=ids, weights=w)
    b = fm.moe_gate(z, 3)
    assert a[0] is ids and a[1] is w and torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    with pytest.raises(ValueError, match="ids"):
        fm.moe_gate(z, 3, ids=ids.long())
    with pytest.raises(ValueError, match="weights"):
        fm.moe_gate(z, 3, weights=w[:20])
    with pytest.raises(ValueError, match="workspace"):
        fm.moe_gate_balance(z, 3, 0.1, workspace=torch.empty(64, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError, match="dlogits"):
        fm.moe_gate_backward(z, a[0], w, dlogits=torch.empty(30, 12, device=DEV, dtype=torch.bfloat16))
    with pytest.raises(fm.Fp8MoeError) as e:
        fm.moe_gate(torch.zeros(2, 1025, device=DEV), 2)
    assert e.value.status == fm._lib.ERR_UNSUPPORTED
    with pytest.raises(ValueError, match="tensors on"):
        fm.moe_gate(z, 3, bias=torch.zeros(12))


def test_repeats_bit_for_bit():
    note("moe_gate_balance repeats")
    z = torch.randn(20000, 48, device=DEV)
    offs = i32_dev([5000, 20000])
    a = fm.moe_gate_balance(z, 5, 0.1, offs)
    for _ in range(3):
        assert all(torch.equal(x, y) for x, y in zip(a, fm.moe_gate_balance(z, 5, 0.1, offs)))


def test_streams_and_graph():
    """On another stream, and captured: replays on new logits give what eager calls give."""
    rng = np.random.default_rng(9)
    T, E, k = 900, 64, 6
    z = torch.randn(T, E, device=DEV)
    offs, bias = i32_dev([300, 850]), 0.1 * torch.randn(E, device=DEV)
    dw = torch.randn(T, k, device=DEV)
    note("gate on a stream and in a graph")

    def step(stream=None):
        a = fm.moe_gate(z, k, fm.GATE_SIGMOID, bias, renormalize=True, stream=stream)
        b = fm.moe_gate_balance(z, k, 0.1, offs, stream=stream)
        c = fm.moe_balance_loss(z, a[0], 0.1, offs, stream=stream)
        d = fm.moe_gate_backward(z, b[0], dw, dprob=b[4], seq_offs=offs, stream=stream)
        e = fm.moe_balance_loss_backward(z, c[2], c[0], offs, stream=stream)
        return (*a, *b, *c, d, e)

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for r in range(4):
        z.copy_(dev(rng.standard_normal((T, E)).astype(np.float32)))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(step(), out)), f"replay {r}"
