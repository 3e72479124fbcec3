"""SwiGLU with its input kept in 8 bits: what is kept bit for bit, results and gradients against fp64 of the kept values, the
MX forms bit for bit against the calls on the same values in bf16, and the run of them in an expert block's step."""
import numpy as np
import pytest
import torch

import mxfp8_quantized_moe_amd as fm
from oracle import codec as oc
from oracle import quant as oq
from oracle import saved as os_
from oracle.quant import bf16_to_f32
from oracle.swiglu import round_bf16
from gpu_helpers import DEV, note, bf16_dev, i32_dev, u8_dev, host, bf16_bits_to_f64, assert_bytes_equal

pytestmark = pytest.mark.gpu

# Row lengths for each kernel: 16, 64 and 256 threads a row, one to eight chunks a thread, and rows read twice.
# (For few rows, that is; the kernels taken from 2048 rows on are in test_gpu_saved_many_rows.py.)
SIZES = [(1, 32), (37, 96), (18, 128), (9, 160), (300, 512), (21, 544), (5, 1056), (66, 1408), (7, 2048), (3, 2080), (4, 4128),
         (2, 8192), (3, 8224), (2, 16384), (2, 16416)]


def inputs(rng, R, F, pad=0):
    h = rng.standard_normal((R, 2 * F + pad)) * np.where(rng.random((R, 2 * F + pad)) < 0.02, 20, 1)
    if R > 2:
        h[R // 2] = 0                    # a row of zeros: a = 0
        h[R // 3] *= 1e-3
    return round_bf16(h)


def amax_between(scale, v, slack, codec):
    """The scale is fmax / the largest magnitude (two fp32 roundings), that magnitude within its slack."""
    fmax = float(oc.FMAX[codec])
    floor = float(np.float32(1e-12))
    lo = fmax / np.maximum((np.abs(v) + slack).max(1), floor) * (1 - 2.0 ** -23)
    hi = fmax / np.maximum((np.abs(v) - slack).max(1), floor) * (1 + 2.0 ** -23)
    s = scale.astype(np.float64)
    assert ((lo <= s) & (s <= hi)).all(), np.argwhere(~((lo <= s) & (s <= hi)))[:3]


def near_bf16(got_bits, v, slack, what):
    """Half a bf16 step (2^-8 of the value at most) over what the fp32 evaluation may be off."""
    got = bf16_bits_to_f64(got_bits)
    off = np.abs(got - v) - (slack + 2.0 ** -8 * (np.abs(v) + slack))
    assert (off <= 0).all(), f"{what}: worst {off.max()} at {np.argwhere(off > 0)[0]}"


@pytest.mark.parametrize("codec,rule,pad", [(0, 0, 0), (1, 1, 40)])
@pytest.mark.parametrize("R,F", SIZES)
def test_save(R, F, codec, rule, pad):
    note(f"swiglu_quantize_rowwise_save {R}x{F} codec {codec} rule {rule} pad {pad}")
    h = inputs(np.random.default_rng(R + F), R, F, pad)
    a2, q, s, hq, hs = fm.swiglu_quantize_rowwise_save(bf16_dev(h)[:, :2 * F], codec=codec, rule=rule, keep_bf16=True)
    h = np.ascontiguousarray(h[:, :2 * F])
    rq, rs = oq.quantize_mx_lastdim(h, rule)
    assert_bytes_equal(host(hs), rs, "kept scales")
    assert_bytes_equal(host(hq), rq, "kept codes")
    a = os_.forward(bf16_to_f32(h).astype(np.float64))
    slack = 10 * 2.0 ** -24 * np.abs(a) + 1e-38
    near_bf16(host(a2), a, slack, "a2")
    amax_between(host(s), a, slack, codec)
    assert os_.between(host(q), host(s), a, slack, codec).all()
    none, q2, s2, hq2, hs2 = fm.swiglu_quantize_rowwise_save(bf16_dev(h), codec=codec, rule=rule)
    assert none is None
    for x, y in ((q, q2), (s, s2), (hq, hq2), (hs, hs2)):
        assert torch.equal(x, y)


@pytest.mark.parametrize("codec", [0, 1])
@pytest.mark.parametrize("R,F", SIZES)
def test_saved_backward(R, F, codec):
    note(f"swiglu_backward_quantize_rowwise_saved {R}x{F} codec {codec}")
    rng = np.random.default_rng(R * F)
    hq, hs = oq.quantize_mx_lastdim(inputs(rng, R, F), codec)
    d = round_bf16(1e-3 * rng.standard_normal((R, F)))
    if R > 2:
        d[R // 2 - 1] = 0
    args = (bf16_dev(d), u8_dev(hq), u8_dev(hs))
    dh1, q, s, a2 = fm.swiglu_backward_quantize_rowwise_saved(*args, codec=codec, want_a2=True)
    h = os_.kept_values(hq, hs)
    dh, slack = os_.backward(bf16_bits_to_f64(d), h)
    near_bf16(host(dh1), dh, slack, "dh1")
    a = os_.forward(h)
    near_bf16(host(a2), a, 10 * 2.0 ** -24 * np.abs(a) + 1e-38, "a2")
    amax_between(host(s), dh, slack, codec)
    assert os_.between(host(q), host(s), dh, slack, codec).all()
    only = fm.swiglu_backward_quantize_rowwise_saved(*args, codec=codec, keep_bf16=False)
    assert only[0] is None and only[3] is None and torch.equal(only[1], q) and torch.equal(only[2], s)
    only = fm.swiglu_backward_quantize_rowwise_saved(*args, codec=codec, codes=False)
    assert only[1] is None and only[2] is None and torch.equal(only[0], dh1)
    only = fm.swiglu_backward_quantize_rowwise_saved(*args, codes=False, keep_bf16=False, want_a2=True)
    assert only[0] is None and torch.equal(only[3], a2)


def test_gradient_by_differences():
    """The kernel's gradient against differences of the kernel-free forward at the kept values."""
    note("swiglu_backward_quantize_rowwise_saved against differences")
    rng = np.random.default_rng(5)
    R, F = 6, 64
    hq, hs = oq.quantize_mx_lastdim(round_bf16(2 * rng.standard_normal((R, 2 * F))), 0)
    d = round_bf16(rng.standard_normal((R, F)))
    dh1 = bf16_bits_to_f64(host(fm.swiglu_backward_quantize_rowwise_saved(bf16_dev(d), u8_dev(hq), u8_dev(hs), codes=False)[0]))
    h, df, eps = os_.kept_values(hq, hs), bf16_bits_to_f64(d), 1e-4
    for half in (0, 1):
        e = np.zeros((1, 2 * F))
        e[:, half * F:(half + 1) * F] = eps       # a column of a depends on its own gate and up alone
        num = (os_.forward(h + e) - os_.forward(h - e)) / (2 * eps) * df
        got = dh1[:, half * F:(half + 1) * F]
        # differences: eps^2 times a third derivative of at most 3 |u|; the bf16 rounding of the result
        lim = 2.0 ** -8 * np.abs(num) + 3e-8 * (1 + np.abs(h).max()) * np.abs(df) + 1e-9
        assert (np.abs(got - num) <= lim).all()


def test_saturated_gates():
    """Gates far from zero: the complement of a sigmoid next to one keeps its digits, none overflows."""
    note("kept SwiGLU saturated gates")
    F = 32
    h = np.zeros((16, 2 * F))
    h[:, :F] = np.linspace(-240, 240, 16)[:, None]
    h[:, F:] = 3
    hq, hs = oq.quantize_mx_lastdim(round_bf16(h), 1)
    d = round_bf16(np.ones((16, F)))
    dh1, q, s, a2 = fm.swiglu_backward_quantize_rowwise_saved(bf16_dev(d), u8_dev(hq), u8_dev(hs), want_a2=True)
    v = os_.kept_values(hq, hs)
    dh, slack = os_.backward(bf16_bits_to_f64(d), v)
    near_bf16(host(dh1), dh, slack, "dh1")
    near_bf16(host(a2), os_.forward(v), 1e-38 + 2.0 ** -20 * np.abs(os_.forward(v)), "a2")


def dual_outputs(R, C, offs, layout):
    rp = fm.quantize_mx_rows_bound(R, len(offs))
    sc = lambda rows, nb: fm.mx_k4_shape(rows, nb) if layout == fm.MX_LAYOUT_K4 else (rows, nb)
    f = lambda shape: torch.full(shape, 0x5A, dtype=torch.uint8, device=DEV)
    return dict(q=f((R, C)), scale=f(sc(R, C // 32)), q_t=f((C, rp)), scale_t=f(sc(C, rp // 32)),
                offs_pad=torch.full((len(offs),), -9, dtype=torch.int32, device=DEV))


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("rule", [0, 1])
@pytest.mark.parametrize("R,F,offs", [(1, 128, [1]), (200, 128, [70, 70, 133, 180]), (130, 384, [0, 130]), (333, 256, [400, 20, 333]),
                                      (64, 1408, [10, 64]), (97, 160, [33, 97])])
def test_mx_forms(R, F, offs, rule, layout):
    note(f"swiglu mx dual saved {R}x{F} offs {offs} rule {rule} layout {layout}")
    rng = np.random.default_rng(R + F)
    hq, hs = oq.quantize_mx_lastdim(inputs(rng, R, F), rule)
    h = bf16_dev(round_bf16(os_.kept_values(hq, hs)))          # eight significant bits: exact
    d = bf16_dev(round_bf16(1e-3 * rng.standard_normal((R, F))))
    od, kw = i32_dev(offs), dict(rule=rule, layout=layout)
    pairs = [(dual_outputs(R, F, offs, layout), fm.swiglu_quantize_mx_dual_saved, (u8_dev(hq), u8_dev(hs), od),
              fm.swiglu_quantize_mx_dual, (h, od), "a2", F)]
    if F % 128 == 0:
        pairs.append((dual_outputs(R, 2 * F, offs, layout), fm.swiglu_backward_quantize_mx_dual_saved,
                      (d, u8_dev(hq), u8_dev(hs), od), fm.swiglu_backward_quantize_mx_dual, (d, h, od), "dh1", 2 * F))
    for out, f, args, ref_f, ref_args, name, C in pairs:
        ref = {k: v.clone() for k, v in out.items()}
        copies = [torch.full((R, C), -3.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
        f(*args, **kw, **out, **{name: copies[0]})
        ref_f(*ref_args, **kw, **ref, **{name: copies[1]})
        for k in out:
            assert torch.equal(out[k], ref[k]), (f.__name__, k)
        assert torch.equal(copies[0], copies[1]), name


def test_every_code_under_every_scale():
    """Gate 256 (its silu is 256 exactly): the activation is 256 times the kept up value, every e4m3 code under every e8m0
    scale up to 2^111, in both recipes. Exact where bf16 is normal; below 2^-126, zero or bf16's spacing."""
    note("kept SwiGLU codes and scales")
    R, F = 239, 256
    hq, hs = np.full((R, 2 * F), 0x78, np.uint8), np.full((R, 2 * F // 32), 127, np.uint8)
    codes = np.arange(256).astype(np.uint8)
    codes[(codes & 0x7F) == 0x7F] = 0                       # the NaN codes
    hq[:, F:], hs[:, F // 32:] = codes, np.arange(R)[:, None]
    want = 256 * np.ldexp(np.tile(oc.decode(codes, 0), (R, 1)), np.arange(R)[:, None] - 127)
    d = bf16_dev(np.zeros((R, F), np.uint16))
    rowwise = fm.swiglu_backward_quantize_rowwise_saved(d, u8_dev(hq), u8_dev(hs), codes=False, want_a2=True)[3]
    mx = torch.empty(R, F, dtype=torch.bfloat16, device=DEV)
    fm.swiglu_quantize_mx_dual_saved(u8_dev(hq), u8_dev(hs), i32_dev([R]), a2=mx)
    for got in (rowwise, mx):
        got = bf16_bits_to_f64(host(got))
        normal = np.abs(want) >= 2.0 ** -118                # the kept value itself normal in bf16
        assert (got[normal] == want[normal]).all()
        assert (np.abs(got - want)[~normal] <= np.maximum(np.abs(want[~normal]), 2.0 ** -125)).all()


def test_no_rows():
    note("kept SwiGLU without rows")
    h = torch.empty(0, 128, dtype=torch.bfloat16, device=DEV)
    a2, q, s, hq, hs = fm.swiglu_quantize_rowwise_save(h, keep_bf16=True)
    assert (a2.shape, q.shape, s.shape, hq.shape, hs.shape) == ((0, 64), (0, 64), (0,), (0, 128), (0, 4))
    out = fm.swiglu_backward_quantize_rowwise_saved(a2, hq, hs, want_a2=True)
    assert out[0].shape == (0, 128) and out[3].shape == (0, 64)


@pytest.mark.parametrize("layout", [fm.MX_LAYOUT_ROWS, fm.MX_LAYOUT_K4])
@pytest.mark.parametrize("saved", [False, True])
def test_backward_without_rows_writes_the_padding(saved, layout):
    """No rows: the columns' form of the whole gradient, 2F of them, is padding."""
    note(f"SwiGLU backward, MX, no rows, saved {saved} layout {layout}")
    F, pad = 128, 256
    da2, offs = torch.empty(0, F, dtype=torch.bfloat16, device=DEV), i32_dev([0, 0])
    q_t = torch.full((2 * F, pad), 0xAB, dtype=torch.uint8, device=DEV)
    sc_t = torch.full((2 * F * pad // 32,), 0xAB, dtype=torch.uint8, device=DEV).view(
        fm.mx_k4_shape(2 * F, pad // 32) if layout == fm.MX_LAYOUT_K4 else (2 * F, pad // 32))
    if saved:
        hq, hs = u8_dev(np.empty((0, 2 * F), np.uint8)), u8_dev(np.empty((0, 2 * F // 32), np.uint8))
        out = fm.swiglu_backward_quantize_mx_dual_saved(da2, hq, hs, offs, rows_pad=pad, q_t=q_t, scale_t=sc_t, layout=layout)
    else:
        h1 = torch.empty(0, 2 * F, dtype=torch.bfloat16, device=DEV)
        out = fm.swiglu_backward_quantize_mx_dual(da2, h1, offs, rows_pad=pad, q_t=q_t, scale_t=sc_t, layout=layout)
    assert out[1].shape == (0, 2 * F)
    assert (q_t == 0).all()
    assert torch.unique(sc_t).numel() == 1 and (sc_t != 0xAB).all()


class Block:
    """An expert block's step in the rowwise recipe whose forward keeps 8 bits of h1 and nothing of a2."""

    def __init__(self, rng, E=3, K=128, F=96, R=150):
        self.E, self.K, self.F, self.R = E, K, F, R
        w1, w2 = round_bf16(0.1 * rng.standard_normal((E, 2 * F, K))), round_bf16(0.1 * rng.standard_normal((E, K, F)))
        self.w1q, self.w1s = fm.quantize_rowwise(bf16_dev(w1.reshape(-1, K)))
        self.w2q, self.w2s = fm.quantize_rowwise(bf16_dev(w2.reshape(-1, F)))
        self.w2tq, self.w2ts = fm.quantize_colwise(bf16_dev(w2))
        self.offs = i32_dev([40, 90, R])

    def mm(self, a, sa, b, sb, N, K):
        return fm.grouped_mm_scaled(fm.GROUPED_M, a, 0, sa, b, 0, sb, fm.SCALE_F32, self.offs, self.E, self.R, N, K)

    def forward(self, x):
        xq, xs = fm.quantize_rowwise(x)
        h1 = self.mm(xq, xs, self.w1q, self.w1s, 2 * self.F, self.K)
        _, q, s, hq, hs = fm.swiglu_quantize_rowwise_save(h1)
        return self.mm(q, s, self.w2q, self.w2s, self.K, self.F), h1, hq, hs

    def backward(self, dy, hq, hs):
        dq, ds = fm.quantize_rowwise(dy)
        da2 = self.mm(dq, ds, self.w2tq, self.w2ts, self.F, self.K)
        dh1, _, _, a2 = fm.swiglu_backward_quantize_rowwise_saved(da2, hq, hs, want_a2=True)
        dyt, dyts = fm.quantize_colwise(dy, self.offs)
        at, ats = fm.quantize_colwise(a2, self.offs)
        ld = at.shape[1]
        dw2 = fm.grouped_mm_scaled(fm.GROUPED_K, dyt, 0, dyts, at, 0, ats, fm.SCALE_F32, self.offs, self.E, ld, self.K, self.F)
        return da2, dh1, a2, dw2


def test_step_of_a_block():
    """Forward and backward through the products: the gradients beside those of the bf16 h1 (what the 8-bit rounding of h1,
    at most half an e4m3 step 2^-4 a value and the FLOOR rule's clamp, leaves of them: a tenth of the norm), and the whole step captured,
    replayed on new inputs between eager steps."""
    note("kept SwiGLU in a block's step")
    rng = np.random.default_rng(8)
    b = Block(rng)
    xs = [bf16_dev(round_bf16(rng.standard_normal((b.R, b.K)))) for _ in range(3)]
    dys = [bf16_dev(round_bf16(1e-2 * rng.standard_normal((b.R, b.K)))) for _ in range(3)]

    def step(x, dy):
        y, h1, hq, hs = b.forward(x)
        return (y, h1, hq, hs) + b.backward(dy, hq, hs)

    y, h1, hq, hs, da2, dh1, a2, dw2 = step(xs[0], dys[0])
    ref_a2 = fm.swiglu_quantize_rowwise(h1, codes=False)[0].float()
    ref_dh = fm.swiglu_backward_quantize_rowwise(da2, h1, codes=False)[0].float()
    for got, ref in ((a2, ref_a2), (dh1, ref_dh)):
        assert float((got.float() - ref).norm() / ref.norm()) < 0.1
    aq, as_ = fm.quantize_rowwise(ref_a2.to(torch.bfloat16))
    ref_y = b.mm(aq, as_, b.w2q, b.w2s, b.K, b.F).float()
    assert float((y.float() - ref_y).norm() / ref_y.norm()) < 0.02   # the forward keeps its own digits
    want = [step(x, d) for x, d in zip(xs, dys)]
    x, dy = xs[0].clone(), dys[0].clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step(x, dy)
    for i in (0, 1, 2, 1):
        x.copy_(xs[i])
        dy.copy_(dys[i])
        g.replay()
        torch.cuda.synchronize()
        for got, ref in zip(out, want[i]):
            assert torch.equal(got.view(torch.uint8), ref.view(torch.uint8))
        step(xs[2], dys[0])
