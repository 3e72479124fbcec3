"""The norm, the gate and the balance loss as they are used together, in front of and behind the routed experts:

  x + residual -> norm (bf16 rows and FP8 codes) -> router logits -> gate and balance loss -> moe_route ->
  moe_permute_quantized -> grouped GEMM -> moe_combine, and back: moe_combine_backward -> gate backward -> norm backward.
"""
import numpy as np
import pytest
import torch

import mxfp8_quantized_moe_amd as fm
from oracle import codec as oc
from oracle import gate as og
from oracle import norm as on
from oracle.swiglu import round_bf16
from gpu_helpers import DEV, note, bf16_dev, i32_dev, host, bf16_bits_to_f64

pytestmark = pytest.mark.gpu

T, C, E, K = 300, 256, 16, 3
EPS, COEF = 1e-6, 0.02


@pytest.fixture(scope="module")
def data():
    rng = np.random.default_rng(21)
    d = dict(x=round_bf16(rng.standard_normal((T, C))), res=round_bf16(2 * rng.standard_normal((T, C))),
             dy=round_bf16(rng.standard_normal((T, C))), dsum=round_bf16(rng.standard_normal((T, C))),
             gamma=(1 + 0.2 * rng.standard_normal(C)).astype(np.float32),
             wr=(rng.standard_normal((E, C)) / 16).astype(np.float32),
             we=round_bf16(rng.standard_normal((E * C, C)) / 16), offs=np.array([130, 290], np.int32))
    return d


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


class Front:
    """One MoE block's front: the user's program around the entry points."""

    def __init__(self, d):
        self.gamma, self.wr, self.offs = dev(d["gamma"]), dev(d["wr"]), i32_dev(d["offs"])
        self.we_q, self.we_s = fm.quantize_rowwise(bf16_dev(d["we"]))
        self.mask = torch.arange(T, device=DEV) % 11 != 0

    def forward(self, x, res):
        h, q, sc, rstd, s = fm.rmsnorm_quantize_rowwise(x, self.gamma, EPS, residual=res)
        logits = h.float() @ self.wr.t()
        ids, w, loss, counts, dprob = fm.moe_gate_balance(logits, K, COEF, self.offs, token_mask=self.mask, renormalize=True,
                                                          route_scale=1.5)
        _, offs, dest, src = fm.moe_route(ids, E, 16)
        qg, sg = fm.moe_permute_quantized(q, sc, src, K)
        yg = fm.grouped_mm_scaled(fm.GROUPED_M, qg, fm.OPD_E4M3FN, sg, self.we_q, fm.OPD_E4M3FN, self.we_s, fm.SCALE_F32,
                                  offs, E, src.numel(), C, C)
        y = fm.moe_combine(yg, dest, w, K)
        return dict(h=h, q=q, sc=sc, rstd=rstd, s=s, logits=logits, ids=ids, w=w, loss=loss, counts=counts, dprob=dprob,
                    dest=dest, src=src, yg=yg, y=y)

    def backward(self, f, dy, dloss, dsum):
        _, _, _, dw = fm.moe_combine_backward(dy, f["yg"], f["dest"], f["src"], f["w"], K, codes=False, rows_out=False)
        dlogits = fm.moe_gate_backward(f["logits"], f["ids"], dw, token_mask=self.mask, renormalize=True, route_scale=1.5,
                                       dprob=f["dprob"], dloss=dloss, seq_offs=self.offs)
        dh = (dlogits @ self.wr).to(torch.bfloat16)
        dx, dgamma = fm.rmsnorm_backward(dh, f["s"], f["rstd"], self.gamma, dsum=dsum)
        return dict(dw=dw, dlogits=dlogits, dx=dx, dgamma=dgamma)


def test_forward(data):
    note("block front, forward")
    m = Front(data)
    f = m.forward(bf16_dev(data["x"]), bf16_dev(data["res"]))
    s_bits = on.residual_sum(data["x"], data["res"])
    assert np.array_equal(host(f["s"]), s_bits)
    mask = host(m.mask)
    logits = host(f["logits"]).astype(np.float64)
    ids, w = og.gate(logits, K, False, None, mask, True, 1.5)
    np.testing.assert_array_equal(host(f["ids"]), ids)
    loss, counts, _ = og.balance(logits, ids, COEF, data["offs"], False, mask)
    np.testing.assert_array_equal(host(f["counts"]), counts)
    assert abs(host(f["loss"])[0] - loss) < 1e-5 * loss
    # the routed experts' outputs: codes of the norm through the grouped GEMM.  FP8 products are exact and their sum is
    # accepted within 2^-10 of the sum of magnitudes (the MFMA's accumulation); yg is bf16, and so is y.
    a = oc.decode(host(f["q"]), 0) / host(f["sc"]).astype(np.float64)[:, None]
    b = (oc.decode(host(m.we_q), 0) / host(m.we_s).astype(np.float64)[:, None]).reshape(E, C, C)
    y = bf16_bits_to_f64(host(f["y"]))
    for t in range(T):
        ref, size = np.zeros(C), np.zeros(C)
        for j in range(K):
            if ids[t, j] >= 0:
                p = b[ids[t, j]] @ a[t]
                ref += w[t, j] * p
                size += w[t, j] * (np.abs(p) * 2.0 ** -8 + 2.0 ** -10 * (np.abs(b[ids[t, j]]) @ np.abs(a[t])) + 1e-5 * np.abs(p))
        assert np.all(np.abs(y[t] - ref) <= size + np.abs(ref) * 2.0 ** -8 + 1e-6), t
    assert np.all(y[~mask] == 0)


def test_backward_is_the_derivative(data):
    """The chain of backward entry points against torch's derivative in 64 bits of
    <dy, sum_j w_j yg_j> + dloss * loss + <dsum, s> with the choices and the experts' outputs fixed."""
    note("block front, backward")
    m = Front(data)
    f = m.forward(bf16_dev(data["x"]), bf16_dev(data["res"]))
    dloss = torch.full((1,), 50.0, device=DEV)
    b = m.backward(f, bf16_dev(data["dy"]), dloss, bf16_dev(data["dsum"]))
    D = torch.float64
    s = torch.from_numpy(bf16_bits_to_f64(host(f["s"]))).requires_grad_(True)
    gamma = torch.from_numpy(data["gamma"].astype(np.float64)).requires_grad_(True)
    wr = torch.from_numpy(data["wr"].astype(np.float64))
    h = s * torch.rsqrt((s * s).mean(1, keepdim=True) + EPS) * gamma
    # the logits' values are those the gate saw (h rounded to bf16); their derivative is the formula's
    z = h @ wr.t()
    z = z + (torch.from_numpy(host(f["logits"]).astype(np.float64)) - z).detach()
    p = torch.softmax(z, 1)
    ids = torch.from_numpy(host(f["ids"]).astype(np.int64))
    on_ = ids >= 0
    u = torch.where(on_, p.gather(1, ids.clamp(min=0)), torch.zeros((), dtype=D))
    w = 1.5 * u / u.sum(1, keepdim=True).clamp(min=1e-300)
    yg, dest = torch.from_numpy(bf16_bits_to_f64(host(f["yg"]))), torch.from_numpy(host(f["dest"]).astype(np.int64)).view(T, K)
    dy = torch.from_numpy(bf16_bits_to_f64(data["dy"]))
    y = (w[:, :, None] * torch.where(on_[:, :, None], yg[dest.clamp(min=0)], torch.zeros((), dtype=D))).sum(1)
    _, _, dprob = og.balance(host(f["logits"]), host(f["ids"]), COEF, data["offs"], False, host(m.mask))
    seq = np.searchsorted(data["offs"], np.arange(T), side="right")
    per = np.concatenate([dprob, np.zeros((1, E))])[seq] * host(m.mask)[:, None]
    total = (dy * y).sum() + 50.0 * (p * torch.from_numpy(per)).sum() \
        + (torch.from_numpy(bf16_bits_to_f64(data["dsum"])) * s).sum()
    gs, gg, gz = torch.autograd.grad(total, [s, gamma, z])
    # dlogits: fp32 throughout from dw, itself an fp32 sum of C exact products: C u of their magnitudes, of which the
    # gradient is a combination with weights u (|dw| + sum |dw| u), so 2 C u of that; 200 u for the gate's own steps
    U = 2.0 ** -24
    size_w = (dy.abs()[:, None, :] * torch.where(on_[:, :, None], yg[dest.clamp(min=0)], torch.zeros((), dtype=D)).abs()).sum(2)
    un = (w / 1.5).detach()
    spread = torch.zeros(T, E, dtype=D).scatter_add_(1, ids.clamp(min=0), 1.5 * un * (size_w + (size_w * un).sum(1, keepdim=True)))
    spread = spread + 2 * 50.0 * p.detach() * torch.from_numpy(per).max(1, keepdim=True).values
    assert bool(((b["dlogits"].double().cpu() - gz).abs() <= (2 * C + 200) * U * spread + 1e-12).all())
    # dh: dlogits @ wr in fp32 (E products), then one rounding to bf16, at most half a step, 2^-8 of its magnitude
    wr_a = wr.abs()
    ddh = 2.0 ** -8 * (gz @ wr).abs() + ((2 * C + 200) * U * spread) @ wr_a + 2 * E * U * (gz.abs() @ wr_a)
    n = (s * torch.rsqrt((s * s).mean(1, keepdim=True) + EPS)).detach()
    dg_tol = (ddh * n.abs()).sum(0) + (T + 50) * U * ((gz @ wr).abs() * n.abs()).sum(0)
    assert bool(((b["dgamma"].double().cpu() - gg).abs() <= 1.01 * dg_tol).all())
    g_tol = ddh * gamma.detach().abs() + 100 * U * (gz @ wr).abs() * gamma.detach().abs()
    rstd = torch.rsqrt((s * s).mean(1, keepdim=True) + EPS).detach()
    dx_tol = rstd * (g_tol + n.abs() * (g_tol * n.abs()).mean(1, keepdim=True)) + 2.0 ** -8 * gs.abs() + 1e-12
    assert bool(((b["dx"].double().cpu() - gs).abs() <= 1.01 * dx_tol).all())


def test_captured(data):
    """Forward and backward in one graph, replayed over new rows with eager work between: every replay equals eager."""
    note("block front, captured")
    m = Front(data)
    x, res, dy, dsum = (bf16_dev(data[n]) for n in ("x", "res", "dy", "dsum"))
    dloss = torch.ones(1, device=DEV)

    def step():
        f = m.forward(x, res)
        return {**f, **m.backward(f, dy, dloss, dsum)}

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for r in range(4):
        rng = np.random.default_rng(60 + r)
        x.copy_(bf16_dev(round_bf16(rng.standard_normal((T, C)))))
        dloss.fill_(1.0 + r)
        graph.replay()
        torch.cuda.synchronize()
        want = m.forward(x, res)
        for n in want:
            if n == "yg":       # rows past the last group are left as they were
                pick = want["dest"][want["dest"] >= 0].long()
                assert pick.numel() and torch.equal(out[n][pick], want[n][pick]), f"replay {r} {n}"
            else:
                assert torch.equal(out[n], want[n]), f"replay {r} {n}"
        # the backward from the replay's own dw (moe_combine_backward sums in an order of its own)
        dz = fm.moe_gate_backward(want["logits"], want["ids"], out["dw"], token_mask=m.mask, renormalize=True, route_scale=1.5,
                                  dprob=want["dprob"], dloss=dloss, seq_offs=m.offs)
        assert torch.equal(out["dlogits"], dz), f"replay {r}"
        dx, dgamma = fm.rmsnorm_backward((dz @ m.wr).to(torch.bfloat16), want["s"], want["rstd"], m.gamma, dsum=dsum)
        assert torch.equal(out["dx"], dx) and torch.equal(out["dgamma"], dgamma), f"replay {r}"


def test_two_streams_at_once(data):
    """Two blocks' fronts interleaved on two streams give what they give alone."""
    note("block front, two streams")
    m = Front(data)
    ins = [(bf16_dev(data["x"]), bf16_dev(data["res"])), (bf16_dev(data["dy"]), bf16_dev(data["x"]))]
    want = [m.forward(*i) for i in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ins]
    got = [None, None]
    for _ in range(5):
        for k, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[k] = m.forward(*ins[k])
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        for n in ("h", "q", "sc", "s", "ids", "w", "loss", "counts", "dprob", "y"):
            assert torch.equal(a[n], b[n]), n
