"""GPU parity of the RMS norm with its 8-bit output and its backward, against the fp64 oracle (oracle/norm.py).

Tolerances, with u = 2^-24 (half an fp32 step).  The sum of squares of one row: a thread adds at most 64 products
(each a fused step), then 4 + 2 lane steps and 2 across waves: at most 72 roundings of positive terms, so 72 u relative.
Mean, eps, square root and division: rstd within (72 + 3) / 2 + 2 < 40 u.  f takes two more products: 42 u, h one bf16
rounding more (2^-8), the rowwise scale one division more (44 u).  A code is the rounding of f * scale (43 u more):
half an e4m3 step, 2^-4 relative for normal values and half the subnormal step (2^-10, fnuz 2^-11) below.
"""
import numpy as np
import pytest
import torch

import mxfp8_quantized_moe_amd as fm
from oracle import codec as oc
from oracle import norm as on
from oracle.quant import bf16_to_f32
from oracle.swiglu import round_bf16
from gpu_helpers import DEV, note, bf16_dev, host, assert_bytes_equal, e8m0_rows_to_k4, bf16_bits_to_f64

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def rows_bits(rng, R, C, outliers=True):
    x = rng.standard_normal((R, C))
    if outliers:
        x = np.where(rng.random((R, C)) < 0.01, x * 40, x)
    return round_bf16(x)


def make_gamma(rng, C, kind):
    if kind is None:
        return None, None
    g = (1 + 0.3 * rng.standard_normal(C)).astype(np.float32)
    if kind == "bf16":
        b = round_bf16(g.astype(np.float64))
        return bf16_dev(b), bf16_bits_to_f64(b)
    return torch.from_numpy(g).to(DEV), g.astype(np.float64)


def strided(bits, pad):
    """bf16 rows as a slice of wider rows whose tail holds NaN (never to be read)."""
    R, C = bits.shape
    wide = np.full((R, C + pad), 0x7FC0, np.uint16)
    wide[:, :C] = bits
    return bf16_dev(wide)[:, :C]


def check_codes(q, y, codec, what):
    """q: codes of values known to within 90 u relative as y (already scaled)."""
    fmax = oc.FMAX[codec]
    sub = 2.0 ** -10 if codec == 0 else 2.0 ** -11
    got = oc.decode(q, codec)
    y = np.clip(y, -fmax, fmax)
    tol = np.maximum(np.abs(y) * 2.0 ** -4, sub) + 90 * U * np.abs(y)
    assert np.all(np.isfinite(got)), what
    assert np.all(np.abs(got - y) <= tol), f"{what}: {np.max(np.abs(got - y) - tol)}"


def check_common(out, s_bits, res, rstd, f, what):
    h, _, _, rs, s = out
    got = host(rs).astype(np.float64)
    assert np.all(np.abs(got - rstd) <= 40 * U * rstd), f"{what} rstd"
    if res is not None:
        assert_bytes_equal(host(s), s_bits, f"{what} sum")
    if h is not None:
        d = np.abs(bf16_bits_to_f64(host(h)) - f)
        assert np.all(d <= np.abs(f) * (2.0 ** -8 + 43 * U) + 2.0 ** -134), f"{what} h"


SHAPES = [(1, 8), (3, 16), (17, 64), (5, 200), (33, 512), (7, 520), (4, 1032), (9, 2048), (2, 2056), (3, 4104), (1, 7168),
          (2, 8200), (5, 16384), (1000, 40), (300, 1000)]


@pytest.mark.parametrize("R,C", SHAPES)
@pytest.mark.parametrize("codec", [0, 1])
def test_rowwise(R, C, codec):
    rng = np.random.default_rng(R * 131 + C + codec)
    kind = (None, "f32", "bf16")[(R + C // 8 + codec) % 3]
    with_res = (R + codec) % 2 == 0
    note(f"rmsnorm_quantize_rowwise {R}x{C} codec {codec} gamma {kind} residual {with_res}")
    x = rows_bits(rng, R, C)
    res = rows_bits(rng, R, C) if with_res else None
    if R > 2:
        x[R // 2] = 0                                     # a row of zeros
        if res is not None:
            res[R // 2] = 0
    gd, gh = make_gamma(rng, C, kind)
    s_bits = on.residual_sum(x, res)
    rstd, f = on.norm(s_bits, gh, 1e-5)
    out = fm.rmsnorm_quantize_rowwise(strided(x, 8), gd, 1e-5, residual=None if res is None else strided(res, 16),
                                      codec=codec)
    check_common(out, s_bits, res, rstd, f, "rowwise")
    scale = host(out[2]).astype(np.float64)
    want = oc.FMAX[codec] / np.maximum(np.abs(f).max(axis=1), 1e-12)
    assert np.all(np.abs(scale - want) <= 44 * U * want)
    check_codes(host(out[1]), f * want[:, None], codec, "rowwise codes")


@pytest.mark.parametrize("R,C", [(1, 32), (3, 64), (17, 96), (5, 224), (33, 512), (7, 544), (4, 2048), (3, 4128), (2, 8192),
                                 (1, 16384), (700, 160)])
@pytest.mark.parametrize("rule", [0, 1])
def test_mx(R, C, rule):
    rng = np.random.default_rng(R * 17 + C + rule)
    note(f"rmsnorm_quantize_mx {R}x{C} rule {rule}")
    x, res = rows_bits(rng, R, C), rows_bits(rng, R, C) if rule else None
    x[0, :32] = 0
    if res is not None:
        res[0, :32] = 0                                   # a block of zeros
    gd, gh = make_gamma(rng, C, "f32")
    s_bits = on.residual_sum(x, res)
    rstd, f = on.norm(s_bits, gh, 1e-6)
    kw = dict(residual=None if res is None else bf16_dev(res), rule=rule)
    out = fm.rmsnorm_quantize_mx(bf16_dev(x), gd, 1e-6, layout=fm.MX_LAYOUT_ROWS, **kw)
    check_common(out, s_bits, res, rstd, f, "mx")
    code = host(out[2])
    amax = np.abs(f).reshape(R, C // 32, 32).max(axis=2)
    lo, hi = (oc.mx_shared_exponent((amax * (1 + t)).astype(np.float32), rule) for t in (-44 * U, 44 * U))
    X = code.astype(np.int64) - 127
    assert np.all((X >= lo) & (X <= hi)), "exponents"
    y = f.reshape(R, C // 32, 32) * np.exp2(-X.astype(np.float64))[:, :, None]
    check_codes(host(out[1]), y.reshape(R, C), 0, "mx codes")
    k4 = fm.rmsnorm_quantize_mx(bf16_dev(x), gd, 1e-6, layout=fm.MX_LAYOUT_K4, **kw)
    assert_bytes_equal(host(k4[1]), host(out[1]), "K4 codes")
    assert_bytes_equal(host(k4[2]), e8m0_rows_to_k4(code), "K4 scales")


def test_more_rows_than_one_launch():
    """2^23 + 5 rows take two launches: the rows around their border against a call on those rows alone."""
    R, C = (1 << 23) + 5, 32
    note("rmsnorm 2^23 + 5 rows")
    x = torch.randn(R, C, device=DEV).to(torch.bfloat16)
    h, q, sc, rs, _ = fm.rmsnorm_quantize_rowwise(x)
    m = fm.rmsnorm_quantize_mx(x, layout=fm.MX_LAYOUT_K4, keep_bf16=False)
    for part in (slice(0, 40), slice((1 << 23) - 20, R)):
        a = fm.rmsnorm_quantize_rowwise(x[part])
        assert all(torch.equal(u[part], v) for u, v in zip((h, q, sc, rs), a))
        b = fm.rmsnorm_quantize_mx(x[part], layout=fm.MX_LAYOUT_K4)
        assert torch.equal(m[1][part], b[1]) and torch.equal(m[2][:, part], b[2])


def test_forms_agree_and_optional_outputs():
    """codes=False / keep_bf16=False change nothing else; the sum may be written over x or the residual."""
    rng = np.random.default_rng(3)
    R, C = 37, 1024
    x, res = bf16_dev(rows_bits(rng, R, C)), bf16_dev(rows_bits(rng, R, C))
    gd, _ = make_gamma(rng, C, "bf16")
    note("rmsnorm optional outputs")
    h, q, sc, rs, s = fm.rmsnorm_quantize_rowwise(x, gd, residual=res)
    a = fm.rmsnorm_quantize_rowwise(x, gd, residual=res, codes=False)
    b = fm.rmsnorm_quantize_rowwise(x, gd, residual=res, keep_bf16=False)
    assert a[1] is None and a[2] is None and b[0] is None
    assert torch.equal(a[0], h) and torch.equal(b[1], q) and torch.equal(b[2], sc) and torch.equal(b[3], rs)
    m = fm.rmsnorm_quantize_mx(x, gd, residual=res)
    assert torch.equal(m[0], h) and torch.equal(m[3], rs) and torch.equal(m[4], s)
    for which in ("x", "res"):
        x2, r2 = x.clone(), res.clone()
        t = x2 if which == "x" else r2
        c = fm.rmsnorm_quantize_rowwise(x2, gd, residual=r2, sum_out=t)
        assert c[4] is t and torch.equal(t, s) and torch.equal(c[1], q) and torch.equal(c[0], h)
    d = fm.rmsnorm_quantize_rowwise(x, gd)
    assert d[4] is x
    with pytest.raises(ValueError, match="sum_out"):
        fm.rmsnorm_quantize_rowwise(x, gd, residual=res, sum_out=torch.empty(R, C + 8, dtype=torch.bfloat16, device=DEV))


def test_a_bad_row_stays_alone():
    rng = np.random.default_rng(4)
    x = rows_bits(rng, 40, 512)
    good = fm.rmsnorm_quantize_rowwise(bf16_dev(x), None)
    x[7, 3], x[21, 100] = 0x7FC0, 0x7F80                   # a NaN and an infinity
    note("rmsnorm rows with NaN and infinity")
    bad = fm.rmsnorm_quantize_rowwise(bf16_dev(x), None)
    keep = torch.tensor([r for r in range(40) if r not in (7, 21)], device=DEV)
    for a, b in zip(good[:4], bad[:4]):
        assert torch.equal(a[keep], b[keep])


def test_empty_and_refused():
    note("rmsnorm empty")
    x = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV)
    h, q, sc, rs, s = fm.rmsnorm_quantize_rowwise(x, None, residual=x.clone())
    assert h.shape == (0, 64) and q.shape == (0, 64) and sc.shape == (0,) and s.shape == (0, 64)
    dx, dg = fm.rmsnorm_backward(x, x, rs)
    assert dx.shape == (0, 64) and torch.equal(dg, torch.zeros(64, device=DEV))
    wide = torch.zeros(2, 16392, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(fm.Fp8MoeError) as e:
        fm.rmsnorm_quantize_rowwise(wide)
    assert e.value.status == fm._lib.ERR_UNSUPPORTED
    with pytest.raises(fm.Fp8MoeError) as e:
        fm.rmsnorm_quantize_rowwise(wide[:, :64], eps=0.0)
    assert e.value.status == fm._lib.ERR_VALUE
    with pytest.raises(ValueError, match="tensors on"):
        fm.rmsnorm_quantize_rowwise(wide[:, :64], torch.ones(64))


def test_workspaces_that_do_not_hold_their_bytes():
    note("rmsnorm_backward, moe_balance_loss workspaces")
    x = torch.ones(40, 64, dtype=torch.bfloat16, device=DEV)
    one = torch.zeros(1, dtype=torch.uint8, device=DEV)
    for bad in (one, one.expand(1 << 20), torch.zeros(1 << 20, dtype=torch.uint8)):
        with pytest.raises(ValueError):
            fm.rmsnorm_backward(x, x, torch.ones(40, device=DEV), workspace=bad)
        with pytest.raises(ValueError, match="workspace"):
            fm.moe_gate_balance(x, 2, 0.1, workspace=bad)


def test_smallest_epsilon():
    """Rows of zeros with an epsilon below the normal fp32 range: rstd stays finite, codes zero."""
    note("rmsnorm smallest epsilon")
    x = torch.zeros(3, 64, dtype=torch.bfloat16, device=DEV)
    for eps in (2.0 ** -149, 2.0 ** -130):
        h, q, sc, rs, _ = fm.rmsnorm_quantize_rowwise(x, eps=eps)
        want = 1.0 / np.sqrt(eps)
        assert np.all(np.abs(host(rs) - want) <= 4 * 2.0 ** -24 * want)   # a root and a quotient, each rounded once
        assert not h.any() and not q.any() and bool(torch.isfinite(sc).all())


BWD = [(1, 8), (2, 48), (17, 64), (5, 200), (70, 512), (7, 520), (33, 2048), (9, 2056), (3, 4104), (2, 8200), (5, 16384),
       (2500, 64), (5000, 600), (1500, 2304)]


@pytest.mark.parametrize("R,C", BWD)
def test_backward(R, C):
    """dx: the products and the mean (at most 64 + 8 roundings of |g n|, plus 4 in its terms) in fp32, one bf16 rounding.
    dgamma: a workgroup adds its rows in turn, then the workgroups' shares: at most R + 16 roundings."""
    rng = np.random.default_rng(R + C)
    kind = (None, "f32", "bf16")[(R + C // 8) % 3]
    with_sum = C % 16 == 0
    note(f"rmsnorm_backward {R}x{C} gamma {kind} dsum {with_sum}")
    s_bits, dh_bits = rows_bits(rng, R, C), round_bf16(1e-3 * rng.standard_normal((R, C)))
    ds_bits = round_bf16(1e-3 * rng.standard_normal((R, C))) if with_sum else None
    gd, gh = make_gamma(rng, C, kind)
    rstd64, _ = on.norm(s_bits, None, 1e-6)
    rstd = rstd64.astype(np.float32)
    s, dh = bf16_bits_to_f64(s_bits), bf16_bits_to_f64(dh_bits)
    ds = None if ds_bits is None else bf16_bits_to_f64(ds_bits)
    dx, dg = on.norm_backward(dh, s, rstd.astype(np.float64), gh, ds)
    sd, dd, rd = bf16_dev(s_bits), bf16_dev(dh_bits), torch.from_numpy(rstd).to(DEV)
    got, gg = fm.rmsnorm_backward(dd, sd, rd, gd, dsum=None if ds is None else bf16_dev(ds_bits))
    g = dh if gh is None else dh * gh
    n = s * rstd[:, None]
    terms = rstd[:, None] * (np.abs(g) + np.abs(n) * np.abs(g * n).mean(axis=1, keepdims=True))
    if ds is not None:
        terms = terms + np.abs(ds)
    err = np.abs(bf16_bits_to_f64(host(got)) - dx)
    assert np.all(err <= np.abs(dx) * 2.0 ** -8 + 80 * U * terms + 2.0 ** -134), "dx"
    assert np.all(np.abs(host(gg) - dg) <= (R + 16) * U * np.abs(dh * n).sum(axis=0) + 1e-38), "dgamma"
    # without dgamma, and in place
    only, none = fm.rmsnorm_backward(dd, sd, rd, gd, dsum=None if ds is None else bf16_dev(ds_bits), want_dgamma=False)
    assert none is None and torch.equal(only, got)
    for which in ("dh", "s", "dsum")[: 2 if ds is None else 3]:
        a = dict(dh=dd.clone(), s=sd.clone(), dsum=None if ds is None else bf16_dev(ds_bits))
        place, dg2 = fm.rmsnorm_backward(rstd=rd, gamma=gd, dx=a[which], **a)
        assert place is a[which] and torch.equal(place, got) and torch.equal(dg2, gg)


def test_backward_repeats_bit_for_bit():
    rng = np.random.default_rng(8)
    s, dh = bf16_dev(rows_bits(rng, 3000, 1000)), bf16_dev(round_bf16(rng.standard_normal((3000, 1000))))
    rstd = torch.rand(3000, device=DEV)
    note("rmsnorm_backward repeats")
    a = fm.rmsnorm_backward(dh, s, rstd)
    for _ in range(3):
        b = fm.rmsnorm_backward(dh, s, rstd)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_streams_and_graph():
    """On another stream, and captured: replays on new data give what eager calls give."""
    rng = np.random.default_rng(9)
    R, C = 600, 2048
    x, res, dh = (bf16_dev(rows_bits(rng, R, C)) for _ in range(3))
    gd, _ = make_gamma(rng, C, "f32")
    note("rmsnorm on a stream and in a graph")

    def step(stream=None):
        f = fm.rmsnorm_quantize_rowwise(x, gd, residual=res, stream=stream)
        m = fm.rmsnorm_quantize_mx(x, gd, residual=res, layout=fm.MX_LAYOUT_K4, stream=stream)
        b = fm.rmsnorm_backward(dh, f[4], f[3], gd, dsum=dh, stream=stream)
        return (*f, *m[:3], *b)

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
    for k in range(4):
        x.copy_(bf16_dev(rows_bits(np.random.default_rng(20 + k), R, C)))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(step(), out)), f"replay {k}"
