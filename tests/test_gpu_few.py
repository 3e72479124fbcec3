"""The whole expert block for a few tokens against fp64, in every weight format, at the sizes and choices where it can go
wrong; against the grouped path on the same quantized weights; captured, on another stream and in place."""
import numpy as np
import pytest
import torch

import mxfp8_quantized_moe_amd as fm
from oracle import few as of
from oracle import codec as oc
from oracle.quant import bf16_to_f32
from oracle.swiglu import round_bf16
from gpu_helpers import DEV, note, bf16_dev, i32_dev, host, bf16_bits_to_f64, e8m0_rows_to_k4

pytestmark = pytest.mark.gpu

FORMATS = ["fp8", "int8", "mx", "mx_k4"]


class Layer:
    """Quantized weights on the GPU and their values in fp64."""

    def __init__(self, rng, E, K, F, fmt, std=0.05):
        self.E, self.K, self.F, self.fmt = E, K, F, fmt
        self.kw = dict(w_fmt=fm.OPD_INT8 if fmt == "int8" else fm.OPD_E4M3FN,
                       scale_kind={"mx": fm.SCALE_E8M0, "mx_k4": fm.SCALE_E8M0_K4}.get(fmt, fm.SCALE_F32))
        self.w1, self.s1, self.v1 = self.quantize(rng, 2 * F, K, std)
        self.w2, self.s2, self.v2 = self.quantize(rng, K, F, std)

    def quantize(self, rng, rows, cols, std):
        w = bf16_dev(round_bf16(std * rng.standard_normal((self.E * rows, cols))))
        if self.fmt.startswith("mx"):
            q, s, _ = fm.quantize_mx(w, layout=fm.MX_LAYOUT_K4 if self.fmt == "mx_k4" else fm.MX_LAYOUT_ROWS)
            code = host(s)
            if self.fmt == "mx_k4":
                code = code.transpose(1, 0, 2).reshape(self.E * rows, -1)[:, :cols // 32]
            v = oc.decode(host(q), 0) * np.repeat(np.ldexp(1.0, code.astype(int) - 127), 32, axis=1)
        else:
            q, s = fm.quantize_rowwise(w, codec=fm.INT8 if self.fmt == "int8" else fm.E4M3FN)
            c = host(q).astype(np.float64) if self.fmt == "int8" else oc.decode(host(q), 0)
            v = c / host(s).astype(np.float64)[:, None]
        return q.view(self.E, rows, cols), s, v.reshape(self.E, rows, cols)

    def __call__(self, x, ids, w, **kw):
        return fm.moe_few_tokens(x, ids, w, self.w1, self.s1, self.w2, self.s2, **self.kw, **kw)

    def check(self, x_bits, ids, w, **kw):
        xd, idd, wd = bf16_dev(x_bits), i32_dev(ids), torch.from_numpy(w).to(DEV)
        out = torch.full((len(ids), self.K), float("nan"), dtype=torch.bfloat16, device=DEV)
        y = self(xd, idd, wd, y=out, **kw)
        assert y is out
        got = bf16_bits_to_f64(host(y))
        ref, bound = of.block(bf16_to_f32(x_bits).astype(np.float64), ids, w.astype(np.float64), self.v1, self.v2)
        bad = ~(np.abs(got - ref) <= bound)
        assert not bad.any(), f"{bad.sum()} of {bad.size} off; worst {np.nanmax(np.abs(got - ref) - bound)} at {np.argwhere(bad)[0]}"
        for _ in range(2):   # the same bits each time
            assert torch.equal(self(xd, idd, wd).view(torch.int16), y.view(torch.int16))
        return y


def choices(rng, T, k, E, kind):
    if kind == "distinct":
        ids = np.stack([rng.permutation(E)[:k] for _ in range(T)])
    elif kind == "one":                       # everybody chooses the same experts
        ids = np.tile(rng.permutation(E)[:k], (T, 1))
    else:                                     # repeated, absent and invalid ids
        ids = rng.integers(-2, E + 2, (T, k))
        ids[0] = ids[0, 0]
        if T > 1:
            ids[T // 2] = -1
    return ids.astype(np.int32), rng.standard_normal((T, k)).astype(np.float32)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,k,E,K,F,kind", [
    (1, 1, 1, 32, 32, "distinct"), (1, 6, 64, 256, 96, "distinct"), (2, 2, 3, 96, 160, "wild"), (5, 3, 7, 1056, 352, "wild"),
    (16, 2, 4, 128, 64, "one"), (17, 1, 5, 192, 128, "one"), (33, 4, 6, 320, 224, "wild"), (64, 8, 40, 512, 256, "distinct"),
    (64, 2, 3, 64, 2080, "one"), (48, 1, 2, 2080, 64, "distinct"), (64, 16, 1024, 64, 32, "wild"), (3, 300, 200, 64, 64, "wild"),
    (20, 2, 2, 7200, 96, "one"), (64, 3, 8, 1824, 928, "wild"), (40, 1, 2, 96, 3616, "distinct"), (64, 1, 1, 7168, 32, "one"),
])
def test_against_fp64(T, k, E, K, F, kind, fmt):
    note(f"moe_few_tokens {fmt} T {T} topk {k} E {E} K {K} F {F} {kind}")
    rng = np.random.default_rng(T * 1000 + K)
    ids, w = choices(rng, T, k, E, kind)
    x = round_bf16(rng.standard_normal((T, K)) * np.where(rng.random((T, K)) < 0.02, 30, 1))
    Layer(rng, E, K, F, fmt).check(x, ids, w)


@pytest.mark.parametrize("fmt", ["fp8", "int8"])
@pytest.mark.parametrize("K,F", [(16, 16), (48, 80), (1040, 336), (144, 1008), (2064, 16)])
def test_steps_that_end_inside(K, F, fmt):
    """K and F multiples of 16 only: the last 64-byte step is partly outside."""
    note(f"moe_few_tokens {fmt} K {K} F {F}")
    rng = np.random.default_rng(K + F)
    ids, w = choices(rng, 7, 2, 3, "distinct")
    Layer(rng, 3, K, F, fmt).check(round_bf16(rng.standard_normal((7, K))), ids, w)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,k,E,K,F", [
    (60, 1, 1, 96, 224), (28, 1, 1, 224, 96), (60, 2, 2, 32, 160),   # more tokens than an instruction's columns
    (64, 2, 2, 96, 7232), (64, 2, 2, 7264, 96), (50, 3, 3, 160, 4832),   # four tiles in the first kernel, the second, the first
])
def test_many_tokens_an_expert(T, k, E, K, F, fmt):
    """Every token's choices differ, so each of E = k experts has all of them; steps that end inside, in each way to load."""
    if fmt in ("fp8", "int8"):
        K, F = K - 16, F - 16
    note(f"moe_few_tokens {fmt} T {T} topk {k} E {E} K {K} F {F}, all tokens at each expert")
    rng = np.random.default_rng(K + F)
    ids, w = choices(rng, T, k, E, "distinct")
    Layer(rng, E, K, F, fmt).check(round_bf16(rng.standard_normal((T, K))), ids, w)


def test_no_expert_no_tokens_no_columns():
    note("moe_few_tokens empty forms")
    rng = np.random.default_rng(1)
    layer = Layer(rng, 4, 64, 32, "fp8")
    ids, w = np.full((6, 2), -1, np.int32), np.ones((6, 2), np.float32)
    y = layer.check(round_bf16(rng.standard_normal((6, 64))), ids, w)
    assert (host(y) == 0).all()
    y = layer(torch.empty(0, 64, dtype=torch.bfloat16, device=DEV), torch.empty(0, 2, dtype=torch.int32, device=DEV),
              torch.empty(0, 2, device=DEV))
    assert y.shape == (0, 64)
    e = torch.empty(4, 0, 64, dtype=torch.uint8, device=DEV)
    y = fm.moe_few_tokens(bf16_dev(round_bf16(rng.standard_normal((6, 64)))), i32_dev(np.ones((6, 2))), torch.ones(6, 2, device=DEV), e,
                          torch.empty(0, device=DEV), e.view(4, 64, 0), torch.ones(4 * 64, device=DEV))
    assert (host(y) == 0).all()


@pytest.mark.parametrize("fmt", ["fp8", "mx"])
def test_rows_apart_and_in_place(fmt):
    """x a slice of wider rows; y written over x; a token's infinity or NaN stays in its own row."""
    note(f"moe_few_tokens {fmt} strided, in place, infinities")
    rng = np.random.default_rng(2)
    T, K, F, E = 9, 128, 96, 3
    layer = Layer(rng, E, K, F, fmt)
    ids, w = choices(rng, T, 2, E, "distinct")
    wide = round_bf16(rng.standard_normal((T, K + 24)))
    idd, wd = i32_dev(ids), torch.from_numpy(w).to(DEV)
    ref = layer.check(np.ascontiguousarray(wide[:, :K]), ids, w)
    assert torch.equal(layer(bf16_dev(wide)[:, :K], idd, wd), ref)
    x = bf16_dev(np.ascontiguousarray(wide[:, :K]))
    assert torch.equal(layer(x, idd, wd, y=x), ref)
    x = bf16_dev(np.ascontiguousarray(wide[:, :K]))
    x[3, K - 1], x[5, 0] = float("inf"), float("nan")
    got = layer(x, idd, wd)
    keep = [t for t in range(T) if t not in (3, 5)]
    assert torch.equal(got[keep], ref[keep])
    assert torch.isnan(got[5]).all() and not torch.isfinite(got[3]).any()


def test_scales_at_the_ends():
    """e8m0 scales from 2^-117 on are exact in bf16; zero blocks carry code 0; large ones keep the sums in range."""
    note("moe_few_tokens extreme e8m0 scales")
    rng = np.random.default_rng(4)
    T, K, F, E = 4, 64, 64, 2
    layer = Layer(rng, E, K, F, "mx")
    s1, s2 = host(layer.s1).copy(), host(layer.s2).copy()
    s1[: F // 2, :] = 10                                       # 2^-117: gates and ups of nearly nothing
    s1[F:F + 8, :] = 127 + 40
    s2[::3, 0] = 10
    s2[1::3, 1] = 127 + 30
    q1, q2 = host(layer.w1).copy(), host(layer.w2).copy()
    q1[0, 5, :32], s1[5, 0] = 0, 0
    layer.w1, layer.s1 = torch.from_numpy(q1).to(DEV), torch.from_numpy(s1).to(DEV)
    layer.s2 = torch.from_numpy(s2).to(DEV)
    dec = lambda q, s, rows, cols: (oc.decode(q, 0).reshape(E * rows, cols) *
                                    np.repeat(np.ldexp(1.0, s.astype(int) - 127), 32, axis=1)).reshape(E, rows, cols)
    layer.v1, layer.v2 = dec(q1, s1, 2 * F, K), dec(q2, s2, K, F)
    ids, w = choices(rng, T, 2, E, "distinct")
    layer.check(round_bf16(rng.standard_normal((T, K))), ids, w)


@pytest.mark.parametrize("k4", [False, True])
def test_every_code_under_every_scale(k4):
    """One token, one expert, one value of the activation that is exactly 1 (gate 256, up 2^-8): y is W2's first column, every
    e4m3 code under every e8m0 scale up to 2^119. Exact where bf16 is normal; below 2^-126, zero or bf16's spacing."""
    note(f"moe_few_tokens MX codes and scales k4 {k4}")
    K, F = 247 * 256, 32
    w1, s1 = np.zeros((1, 2 * F, K), np.uint8), np.zeros((2 * F, K // 32), np.uint8)
    w1[0, 0, 0], s1[0, 0] = 0x78, 127                       # 256
    w1[0, F, 0], s1[F, 0] = 0x38, 119                       # 2^-8
    codes, scales = np.tile(np.arange(256), 247).astype(np.uint8), np.repeat(np.arange(247), 256).astype(np.uint8)
    codes[(codes & 0x7F) == 0x7F] = 0                       # the NaN codes
    w2 = np.zeros((1, K, F), np.uint8)
    w2[0, :, 0] = codes
    lay = e8m0_rows_to_k4 if k4 else (lambda v: v)
    dev = lambda v: torch.from_numpy(np.ascontiguousarray(v)).to(DEV)
    x = np.zeros((1, K), np.uint16)
    x[0, 0] = 0x3F80
    y = fm.moe_few_tokens(bf16_dev(x), i32_dev([[0]]), torch.ones(1, 1, device=DEV), dev(w1), dev(lay(s1)), dev(w2),
                          dev(lay(scales[:, None])), scale_kind=fm.SCALE_E8M0_K4 if k4 else fm.SCALE_E8M0)
    got = bf16_bits_to_f64(host(y))[0]
    want = np.ldexp(oc.decode(codes, 0), scales.astype(int) - 127)
    normal = np.abs(want) >= 2.0 ** -126
    assert (got[normal] == want[normal]).all()
    assert (np.abs(got - want)[~normal] <= np.maximum(np.abs(want[~normal]), 2.0 ** -133)).all()


def test_every_whole_number():
    """The same with integer weights: every byte, -128 among them."""
    note("moe_few_tokens int8 bytes")
    K, F = 256, 16
    w1, w2 = np.zeros((1, 2 * F, K), np.int8), np.zeros((1, K, F), np.int8)
    w1[0, 0, 0], w1[0, F, 0] = 64, 1
    w2[0, :, 0] = np.arange(-128, 128)
    s1, s2 = np.ones((1, 2 * F), np.float32), np.ones((1, K), np.float32)
    s1[0, F] = 64
    dev = lambda v: torch.from_numpy(np.ascontiguousarray(v)).to(DEV)
    x = np.zeros((1, K), np.uint16)
    x[0, 0] = 0x3F80
    y = fm.moe_few_tokens(bf16_dev(x), i32_dev([[0]]), torch.ones(1, 1, device=DEV), dev(w1), dev(s1), dev(w2), dev(s2),
                          w_fmt=fm.OPD_INT8)
    assert (bf16_bits_to_f64(host(y))[0] == np.arange(-128, 128)).all()


def test_what_must_not_be_read():
    """NaN in experts nobody chose, in weights of slots without an expert and all over the workspace reaches no output; one
    workspace serves calls of different sizes one after the other."""
    note("moe_few_tokens workspace and unread NaN")
    rng = np.random.default_rng(11)
    E, K, F = 6, 96, 64
    layer = Layer(rng, E, K, F, "fp8")
    q1, q2 = layer.w1.clone(), layer.w2.clone()
    q1[4:], q2[4:] = 0x7F, 0x7F
    layer.w1, layer.w2 = q1, q2
    ws = torch.full((fm.moe_few_tokens_workspace_bytes(64, 8, K, F),), 0xFF, dtype=torch.uint8, device=DEV)
    for T, k, kind in [(64, 8, "wild"), (3, 2, "distinct"), (40, 1, "one"), (1, 8, "wild"), (64, 8, "wild")]:
        ids, w = choices(rng, T, k, 4, kind) if kind != "wild" else (rng.integers(-2, 4, (T, k)).astype(np.int32),
                                                                    rng.standard_normal((T, k)).astype(np.float32))
        w = np.where(ids < 0, np.float32("nan"), w).astype(np.float32)
        ref_w = np.where(ids < 0, 0, w).astype(np.float32)
        x = bf16_dev(round_bf16(rng.standard_normal((T, K))))
        y = layer(x, i32_dev(ids), torch.from_numpy(w).to(DEV), workspace=ws)
        ref = layer(x, i32_dev(ids), torch.from_numpy(ref_w).to(DEV))
        assert torch.isfinite(y).all() and torch.equal(y, ref)


@pytest.mark.parametrize("fmt", ["fp8", "int8"])
def test_beside_the_grouped_path(fmt):
    """A decoding step and a prompt's path over the same weights: the few tokens' answer within what the grouped path's
    quantized activations and bf16 intermediates leave (e4m3 half a step 2^-4 an element, int8 2^-1 / 127 of the row's
    largest; both enter twice, as random signs over hundreds of terms: under a tenth of the norm)."""
    note(f"moe_few_tokens {fmt} beside moe_route .. moe_combine")
    rng = np.random.default_rng(6)
    T, k, E, K, F = 24, 2, 4, 256, 320
    layer = Layer(rng, E, K, F, fmt)
    x = bf16_dev(round_bf16(rng.standard_normal((T, K))))
    ids, w = fm.moe_gate(torch.randn(T, E, device=DEV, generator=torch.Generator(DEV).manual_seed(1)), k, renormalize=True)
    codec, opd = (fm.INT8, fm.OPD_INT8) if fmt == "int8" else (fm.E4M3FN, fm.OPD_E4M3FN)
    _, offs, dest, src = fm.moe_route(ids, E, 16)
    R = src.numel()
    _, qg, sg = fm.moe_permute_rowwise(x, src, k, codec=codec)
    h1 = fm.grouped_mm_scaled(fm.GROUPED_M, qg, opd, sg, layer.w1, opd, layer.s1, fm.SCALE_F32, offs, E, R, 2 * F, K)
    _, qa, sa = fm.swiglu_quantize_rowwise(h1, codec=codec)
    yg = fm.grouped_mm_scaled(fm.GROUPED_M, qa, opd, sa, layer.w2, opd, layer.s2, fm.SCALE_F32, offs, E, R, K, F)
    ref = fm.moe_combine(yg, dest, w, k).float()
    got = layer(x, ids, w).float()
    assert float((got - ref).norm() / ref.norm()) < 0.1


def test_captured_and_side_by_side():
    """Two graphs with a workspace each, replayed side by side on two streams, eager calls between."""
    note("moe_few_tokens captured")
    rng = np.random.default_rng(7)
    T, k, E, K, F = 12, 3, 8, 512, 256
    layer = Layer(rng, E, K, F, "fp8")
    inputs = []
    for _ in range(3):
        ids, w = choices(rng, T, k, E, "distinct")
        inputs.append((bf16_dev(round_bf16(rng.standard_normal((T, K)))), i32_dev(ids), torch.from_numpy(w).to(DEV)))
    want = [layer(*v) for v in inputs]
    streams, graphs = [torch.cuda.Stream(), torch.cuda.Stream()], []
    torch.cuda.synchronize()
    for s in streams:
        held = [t.clone() for t in inputs[0]]
        ws = torch.empty(fm.moe_few_tokens_workspace_bytes(T, k, K, F), dtype=torch.uint8, device=DEV)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            y = layer(*held, workspace=ws)
        graphs.append((g, held, y))
    for round_ in range(4):
        order = [(round_ + i) % 3 for i in range(2)]
        for (g, held, y), n in zip(graphs, order):
            for a, b in zip(held, inputs[n]):
                a.copy_(b)
        torch.cuda.synchronize()
        for (g, _, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        eager = layer(*inputs[2], stream=streams[1])
        torch.cuda.synchronize()
        for (_, _, y), n in zip(graphs, order):
            assert torch.equal(y, want[n])
        assert torch.equal(eager, want[2])
