"""Timed cases of the operators in front of an MoE layer's routed path: the RMS norm with the residual's addition and an
8-bit output, the router gate, and the balance loss, each with its backward pass.

``run`` computes a case in plain torch operations, or, with ``own`` set, through the package's entry points; ``exact`` gives
the same outputs from the definitions in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
F8 = {"e4m3fn": (torch.float8_e4m3fn, 448.0, 0), "e4m3fnuz": (torch.float8_e4m3fnuz, 240.0, 1)}
FLT_MAX = torch.finfo(torch.float32).max

MOST_NORM = 16384 * 5120     # elements of the largest norm
MOST_GATE = 65536 * 256      # logits of the largest gate


# ---------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # serving, one token for each of 16 sequences in front of DeepSeek-V3-sized experts: latency
        dict(name="norm_decode", op="norm", form="rowwise", codec="e4m3fn", rows=16, cols=7168, residual=True, gamma="f32",
             keep=True, pad=0),
        # the norm in front of a Llama3-8B linear layer: codes for its forward GEMM, h for its weight gradient
        dict(name="norm_llama3_8b", op="norm", form="rowwise", codec="e4m3fn", rows=8192, cols=4096, residual=True,
             gamma="bf16", keep=True, pad=0),
        # Llama4-Scout's token rows in the MXFP8 recipe
        dict(name="norm_scout_mx", op="norm", form="mx", rule="floor", layout="k4", rows=16384, cols=5120, residual=True,
             gamma="f32", keep=True, pad=0),
        # odd sizes: a slice of wider rows, no residual, the fnuz codec, codes only
        dict(name="norm_odd", op="norm", form="rowwise", codec="e4m3fnuz", rows=4093, cols=2056, residual=False, gamma="bf16",
             keep=False, pad=24),
        # a short micro-batch of DeepSeek-MoE-16B rows
        dict(name="norm_bwd_short", op="norm_backward", rows=509, cols=2048, dsum=False, gamma="f32"),
        # Llama4-Scout's token rows, the residual stream's gradient added
        dict(name="norm_bwd_scout", op="norm_backward", rows=16384, cols=5120, dsum=True, gamma="f32"),
        # serving: 16 tokens over 64 experts
        dict(name="gate_decode", op="gate", tokens=16, experts=64, topk=6, score="softmax", dtype="f32", bias=False,
             renorm=False, scale=1.0, mask=False, dead=False),
        # many experts with a selection bias, sigmoid scores normalised over the chosen ones
        dict(name="gate_wide", op="gate", tokens=65536, experts=256, topk=8, score="sigmoid", dtype="f32", bias=True,
             renorm=True, scale=2.5, mask=False, dead=False),
        # DeepSeek-MoE-16B's gate (64 experts, top 6) with the loss over four sequences
        dict(name="gate_balance_16b", op="gate_balance", tokens=8192, experts=64, topk=6, score="softmax", dtype="f32",
             bias=False, renorm=False, scale=1.0, mask=False, dead=False, seqs=4),
        # Llama4-Scout's 16 experts, top 1, bf16 logits of a padded batch: the loss of choices made before
        dict(name="balance_scout", op="balance", tokens=16384, experts=16, topk=1, score="sigmoid", dtype="bf16", mask=True,
             dead=False, seqs=8),
        # the gradient of both into DeepSeek-MoE-16B's router logits
        dict(name="gate_bwd_16b", op="gate_backward", tokens=8192, experts=64, topk=6, score="softmax", dtype="f32",
             renorm=False, scale=1.0, mask=False, dead=False, seqs=4, gate=True),
        dict(name="gate_bwd_wide", op="gate_backward", tokens=65536, experts=256, topk=8, score="sigmoid", dtype="f32",
             renorm=True, scale=2.5, mask=True, dead=False, seqs=1, gate=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_backward", "gate", "gate_balance", "balance", "gate_backward"])
    if op.startswith("norm"):
        mx = op == "norm" and rng.random() < 0.5
        step = 32 if mx else 8
        cols = step * _log_int(rng, 2, 16384 // step)
        rows = _log_int(rng, 1, max(1, min(16384, MOST_NORM // cols)))
        case = dict(op=op, rows=rows, cols=cols, gamma=rng.choice(["f32", "bf16", "none"]))
        if op == "norm_backward":
            return dict(case, dsum=rng.random() < 0.5)
        case |= dict(residual=rng.random() < 0.7, keep=rng.random() < 0.7, pad=rng.choice([0, 8, 40]))
        if mx:
            return dict(case, form="mx", rule=rng.choice(["floor", "ceil"]), layout=rng.choice(["rows", "k4"]))
        return dict(case, form="rowwise", codec=rng.choice(["e4m3fn", "e4m3fnuz"]))
    experts = _log_int(rng, 2, 1024)
    tokens = _log_int(rng, 1, min(65536, MOST_GATE // experts))
    case = dict(op=op, tokens=tokens, experts=experts, topk=rng.randint(1, min(experts, 12)),
                score=rng.choice(["softmax", "sigmoid"]), dtype=rng.choice(["f32", "f32", "bf16"]),
                mask=rng.random() < 0.4 and tokens >= 32, dead=rng.random() < 0.3)
    if op != "balance":
        case |= dict(renorm=rng.random() < 0.5, scale=rng.choice([1.0, 2.5]))
    if op in ("gate", "gate_balance"):
        case |= dict(bias=rng.random() < 0.4)
    if op != "gate":
        case |= dict(seqs=rng.choice([1, 1, 3, 16, 61]))
    if op == "gate_backward":
        case |= dict(gate=rng.random() < 0.8)
        if not case["gate"]:   # with every eligible expert chosen the loss is constant: no gradient to compare
            case |= dict(topk=min(case["topk"], experts // 2), dead=False)
    return case


def work(case):
    if case["op"] == "norm":
        n = case["rows"] * case["cols"]
        b = 2 + (4 if case["residual"] else 0) + (2 if case["keep"] else 0) + 1 + (1 / 32 if case["form"] == "mx" else 0)
        return {"bytes": n * b + 8 * case["rows"] + 4 * case["cols"], "flops": 10 * n}
    if case["op"] == "norm_backward":
        n = case["rows"] * case["cols"]
        return {"bytes": n * (8 if case["dsum"] else 6) + 4 * case["rows"] + 8 * case["cols"], "flops": 12 * n}
    n, slots = case["tokens"] * case["experts"], case["tokens"] * case["topk"]
    elem = 4 if case["dtype"] == "f32" else 2
    stats = 8 * case.get("seqs", 0) * case["experts"]
    rows = case["tokens"] if case["mask"] else 0
    if case["op"] == "gate_backward":
        return {"bytes": 2 * n * elem + (8 * slots if case["gate"] else 0) + stats / 2 + rows, "flops": 12 * n}
    return {"bytes": n * elem + (4 if case["op"] == "balance" else 8) * slots + stats + rows, "flops": 8 * n}


# ---------------------------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _rows(g, rows, cols, pad=0, sigma=1.0):
    """bf16 activations with 1% outliers, a slice of rows `pad` elements wider."""
    x = torch.randn(rows, cols + pad, generator=g, device=DEV) * sigma
    x = torch.where(torch.rand(rows, cols + pad, generator=g, device=DEV) < 0.01, x * 30, x)
    return x.to(torch.bfloat16)[:, :cols]


def _gamma(g, cols, kind):
    if kind == "none":
        return None
    return (1 + 0.2 * torch.randn(cols, generator=g, device=DEV)).to(torch.float32 if kind == "f32" else torch.bfloat16)


def _logits(g, case):
    """Router logits: experts of unequal popularity; `dead`: some experts masked out with the lowest value, some rows wholly."""
    T, E = case["tokens"], case["experts"]
    z = torch.randn(T, E, generator=g, device=DEV) * 1.5 + torch.randn(E, generator=g, device=DEV) * 0.5
    if case["dead"]:
        gone = torch.rand(T, E, generator=g, device=DEV) < 0.2
        gone |= torch.rand(T, 1, generator=g, device=DEV) < 0.02
        z = torch.where(gone, -math.inf, z)
    return z.to(torch.float32 if case["dtype"] == "f32" else torch.bfloat16)


def _seq_offs(g, case):
    """Inclusive ends of the batch's sequences, of unequal lengths; with a mask a few rows belong to none."""
    S, T = case["seqs"], case["tokens"]
    last = T - T // 37 if case["mask"] else T
    inner = torch.sort(torch.randint(0, last + 1, (S - 1,), generator=g, device=DEV)).values
    return torch.cat([inner, torch.tensor([last], device=DEV)]).to(torch.int32)


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=case)
    if case["op"] == "norm":
        s["x"] = _rows(g, case["rows"], case["cols"], case["pad"])
        s["residual"] = _rows(g, case["rows"], case["cols"], case["pad"], 2.0) if case["residual"] else None
        s["gamma"] = _gamma(g, case["cols"], case["gamma"])
        return s
    if case["op"] == "norm_backward":
        s["s"] = _rows(g, case["rows"], case["cols"])
        s["gamma"] = _gamma(g, case["cols"], case["gamma"])
        s["dh"] = (1e-3 * torch.randn(case["rows"], case["cols"], generator=g, device=DEV)).to(torch.bfloat16)
        s["dsum"] = (1e-3 * torch.randn(case["rows"], case["cols"], generator=g, device=DEV)).to(torch.bfloat16) \
            if case["dsum"] else None
        s["rstd"] = torch.rsqrt(s["s"].float().square().mean(1) + EPS)
        return s
    s["logits"] = _logits(g, case)
    s["mask"] = (torch.rand(case["tokens"], generator=g, device=DEV) < 0.9).to(torch.uint8) if case["mask"] else None
    s["bias"] = 0.1 * torch.randn(case["experts"], generator=g, device=DEV) if case.get("bias") else None
    if case["op"] != "gate":
        s["seq_offs"] = _seq_offs(g, case)
    if case["op"] in ("balance", "gate_backward"):
        s["ids"] = _choose(_eligible(s["logits"].float()), s["mask"], case["topk"]).to(torch.int32)
    if case["op"] == "gate_backward":
        s["dweights"] = 1e-3 * torch.randn(case["tokens"], case["topk"], generator=g, device=DEV) if case["gate"] else None
        _, _, s["dprob"] = _plain_balance(s["logits"], s["ids"], s["mask"], s["seq_offs"], case["score"])
        s["dloss"] = 0.5 + torch.rand(1, generator=g, device=DEV)
    return s


# ---------------------------------------------------------------------------------------------- plain forms

EPS = 1e-6
COEF = 0.01


def _plain_norm(st):
    case, x, res, gamma = st["case"], st["x"], st["residual"], st["gamma"]
    s = x if res is None else (x.float() + res.float()).to(torch.bfloat16)
    v = s.float()
    rstd = torch.rsqrt(v.square().mean(1) + EPS)
    f = v * rstd[:, None]
    if gamma is not None:
        f = f * gamma.float()
    out = {"rstd": rstd}
    if res is not None:
        out["sum"] = s
    if case["keep"]:
        out["h"] = f.to(torch.bfloat16)
    if case["form"] == "rowwise":
        dt, fmax, _ = F8[case["codec"]]
        scale = fmax / f.abs().amax(1).clamp(min=1e-12)
        out["q"], out["scale"] = (f * scale[:, None]).clamp(-fmax, fmax).to(dt), scale
        return out
    blocks = f.view(f.shape[0], -1, 32)
    X = _mx_exponent(blocks.abs().amax(2), case["rule"])
    out["q"] = (blocks * torch.exp2(-X.float())[:, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(f.shape)
    code = (X + 127).to(torch.uint8)
    out["scale"] = (_k4(code) if case["layout"] == "k4" else code).view(torch.float8_e8m0fnu)
    return out


def _mx_exponent(amax, rule):
    """floor(log2 amax) - 8, one more under the CEIL rule where the significand is over 1.75; -127 for a zero block."""
    m, e = torch.frexp(amax)                       # amax = m 2^e, m in [0.5, 1)
    X = e - 9 + ((m > 0.875).to(e.dtype) if rule == "ceil" else 0)
    return torch.where(amax == 0, -127, X.clamp(-127, 127))


def _k4(code):
    """Row-major scale bytes [R, NB] as [ceil(NB / 4), R, 4]."""
    R, NB = code.shape
    G = -(-NB // 4)
    p = torch.zeros(R, 4 * G, dtype=torch.uint8, device=code.device)
    p[:, :NB] = code
    return p.view(R, G, 4).permute(1, 0, 2).contiguous()


def _plain_norm_backward(st):
    s, dh, rstd, gamma, dsum = st["s"].float(), st["dh"].float(), st["rstd"], st["gamma"], st["dsum"]
    n = s * rstd[:, None]
    g = dh if gamma is None else dh * gamma.float()
    dx = rstd[:, None] * (g - n * (g * n).mean(1, keepdim=True))
    if dsum is not None:
        dx = dx + dsum.float()
    return {"dx": dx.to(torch.bfloat16), "dgamma": (dh * n).sum(0)}


def _eligible(z):
    """Logits as the gate reads them: NaN as -inf, at most the largest finite value."""
    return torch.where(torch.isnan(z), -math.inf, z).clamp(max=FLT_MAX)


def _scores(z, kind):
    """Scores of the eligible experts (0 elsewhere), in z's type."""
    if kind == "sigmoid":
        return torch.sigmoid(z)
    e = torch.exp(z - z.amax(1, keepdim=True).clamp(min=-FLT_MAX))
    return e / e.sum(1, keepdim=True).clamp(min=1e-30)


def _choose(key, mask, topk):
    """The topk highest keys in decreasing order, ties to the lower index; -1 where no eligible expert (or token) is left."""
    val, idx = torch.sort(key, dim=1, descending=True, stable=True)
    gone = val[:, :topk] == -math.inf
    if mask is not None:
        gone = gone | (mask == 0)[:, None]
    return torch.where(gone, -1, idx[:, :topk])


def _plain_gate(st):
    case = st["case"]
    z = _eligible(st["logits"].float())
    key = z
    if st["bias"] is not None:   # scores next to each other decide here: 64 bits
        key = torch.where(z > -math.inf, _scores(z.double(), case["score"]) + st["bias"].double(), -math.inf)
    ids = _choose(key, st["mask"], case["topk"])
    w = torch.where(ids >= 0, _scores(z, case["score"]).gather(1, ids.clamp(min=0)), 0.0)
    if case["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    return {"ids": ids.to(torch.int32), "weights": w * case["scale"]}


def _segments(seq_offs, mask, T):
    """Each token's sequence (the count of sequences behind the last one), and whether the token counts."""
    end = torch.cummax(seq_offs.long().clamp(0, T), 0).values
    of = torch.searchsorted(end, torch.arange(T, device=end.device), right=True)
    counts = of < end.numel()
    if mask is not None:
        counts = counts & (mask != 0)
    return of, counts


def _share(z, kind):
    """What the loss averages: scores that sum to 1 over a token's eligible experts."""
    s = _scores(z, kind)
    return s if kind == "softmax" else s / s.sum(1, keepdim=True).clamp(min=1e-30)


def _plain_balance(logits, ids, mask, seq_offs, score):
    T, E = logits.shape
    S, k = seq_offs.numel(), ids.shape[1]
    of, valid = _segments(seq_offs, mask, T)
    member = ((torch.arange(S, device=of.device)[:, None] == of) & valid).double()   # [S, T]: sums over tokens in 64 bits
    n = member.sum(1, keepdim=True)
    P = member @ _share(_eligible(logits.float()), score).double() / n.clamp(min=1)
    ok = valid[:, None] & (ids >= 0)
    at = torch.where(ok, of[:, None] * E + ids, S * E).reshape(-1)
    counts = torch.zeros(S * E + 1, dtype=torch.int32, device=logits.device).scatter_add_(0, at, torch.ones_like(at, dtype=torch.int32))
    counts = counts[:-1].view(S, E)
    f = counts.double() * E / (k * n.clamp(min=1))
    loss = (COEF / S * (f * P).sum()).float().view(1)
    return loss, counts, (COEF / S * f / n.clamp(min=1)).float()


def _plain_gate_backward(st):
    case = st["case"]
    z = _eligible(st["logits"].float())
    s = _scores(z, case["score"])
    of, valid = _segments(st["seq_offs"], st["mask"], z.shape[0])
    dprob = torch.cat([st["dprob"], st["dprob"].new_zeros(1, z.shape[1])])
    dp = torch.where(valid[:, None], dprob[of] * st["dloss"], 0.0)
    if case["score"] == "sigmoid":   # the loss takes s over its sum
        total = s.sum(1, keepdim=True).clamp(min=1e-30)
        dp = (dp - (dp * s / total).sum(1, keepdim=True)) / total
    if case["gate"]:
        ids = st["ids"].long()
        ok, at = ids >= 0, ids.clamp(min=0)
        dw = torch.where(ok, st["dweights"] * case["scale"], 0.0)
        w = torch.where(ok, s.gather(1, at), 0.0)
        if case["renorm"]:
            total = w.sum(1, keepdim=True)
            u = w / total.clamp(min=1e-30)
            dw = torch.where(ok & (total > 0), (dw - (dw * u).sum(1, keepdim=True)) / total.clamp(min=1e-30), 0.0)
        dp = dp.scatter_add(1, at, dw)
    if case["score"] == "sigmoid":
        dz = dp * s * (1 - s)
    else:
        dz = s * (dp - (dp * s).sum(1, keepdim=True))
    if st["mask"] is not None:
        dz = torch.where((st["mask"] != 0)[:, None], dz, 0.0)
    return {"dlogits": dz.to(st["logits"].dtype)}


# ---------------------------------------------------------------------------------------------- one pass

def run(st):
    case, op = st["case"], st["case"]["op"]
    if own:
        return _own(st)
    if op == "norm":
        return _plain_norm(st)
    if op == "norm_backward":
        return _plain_norm_backward(st)
    if op == "gate":
        return _plain_gate(st)
    if op == "gate_backward":
        return _plain_gate_backward(st)
    out = _plain_gate(st) if op == "gate_balance" else {}
    loss, counts, dprob = _plain_balance(st["logits"], out.get("ids", st.get("ids")), st["mask"], st["seq_offs"], case["score"])
    return out | {"loss": loss, "counts": counts, "dprob": dprob}


def _own(st):
    import mxfp8_quantized_moe_amd as fm
    case, op = st["case"], st["case"]["op"]
    if op == "norm":
        if case["form"] == "rowwise":
            dt, _, codec = F8[case["codec"]]
            h, q, scale, rstd, s = fm.rmsnorm_quantize_rowwise(st["x"], st["gamma"], EPS, residual=st["residual"], codec=codec,
                                                               keep_bf16=case["keep"])
            out = {"rstd": rstd, "q": q.view(dt), "scale": scale}
        else:
            h, q, scale, rstd, s = fm.rmsnorm_quantize_mx(
                st["x"], st["gamma"], EPS, residual=st["residual"], keep_bf16=case["keep"],
                rule=fm.MX_CEIL if case["rule"] == "ceil" else fm.MX_FLOOR_OCP,
                layout=fm.MX_LAYOUT_K4 if case["layout"] == "k4" else fm.MX_LAYOUT_ROWS)
            out = {"rstd": rstd, "q": q.view(torch.float8_e4m3fn), "scale": scale.view(torch.float8_e8m0fnu)}
        if case["residual"]:
            out["sum"] = s
        if case["keep"]:
            out["h"] = h
        return out
    if op == "norm_backward":
        dx, dgamma = fm.rmsnorm_backward(st["dh"], st["s"], st["rstd"], st["gamma"], dsum=st["dsum"])
        return {"dx": dx, "dgamma": dgamma}
    score = fm.GATE_SIGMOID if case["score"] == "sigmoid" else fm.GATE_SOFTMAX
    if op == "gate":
        ids, weights = fm.moe_gate(st["logits"], case["topk"], score=score, bias=st["bias"], token_mask=st["mask"],
                                   renormalize=case["renorm"], route_scale=case["scale"])
        return {"ids": ids, "weights": weights}
    if op == "gate_balance":
        ids, weights, loss, counts, dprob = fm.moe_gate_balance(
            st["logits"], case["topk"], COEF, seq_offs=st["seq_offs"], score=score, bias=st["bias"], token_mask=st["mask"],
            renormalize=case["renorm"], route_scale=case["scale"])
        return {"ids": ids, "weights": weights, "loss": loss, "counts": counts, "dprob": dprob}
    if op == "balance":
        loss, counts, dprob = fm.moe_balance_loss(st["logits"], st["ids"], COEF, seq_offs=st["seq_offs"], score=score,
                                                  token_mask=st["mask"])
        return {"loss": loss, "counts": counts, "dprob": dprob}
    if not case["gate"]:
        return {"dlogits": fm.moe_balance_loss_backward(st["logits"], st["dprob"], dloss=st["dloss"], seq_offs=st["seq_offs"],
                                                        score=score, token_mask=st["mask"])}
    return {"dlogits": fm.moe_gate_backward(st["logits"], st["ids"], st["dweights"], score=score, token_mask=st["mask"],
                                            renormalize=case["renorm"], route_scale=case["scale"], dprob=st["dprob"],
                                            dloss=st["dloss"], seq_offs=st["seq_offs"])}


# ---------------------------------------------------------------------------------------------- definitions in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    D = torch.float64
    if case["op"] == "norm":
        s = st["x"].to(D)
        if case["residual"]:
            s = (s + st["residual"].to(D)).to(torch.bfloat16).to(D)   # the stream is bf16 by definition
        rstd = 1 / torch.sqrt((s * s).sum(1) / case["cols"] + EPS)
        f = torch.einsum("rc,r->rc", s, rstd)
        if st["gamma"] is not None:
            f *= st["gamma"].to(D)
        out = {"rstd": rstd}
        if case["residual"]:
            out["sum"] = s
        if case["keep"]:
            out["h"] = f
        if case["form"] == "rowwise":
            fmax = F8[case["codec"]][1]
            out["scale"] = fmax / torch.maximum(f.abs().max(1).values, torch.tensor(1e-12, dtype=D, device=DEV))
            out["q"] = f * out["scale"][:, None]
            return out
        b = f.reshape(case["rows"], case["cols"] // 32, 32)
        a = b.abs().max(2).values
        lg = torch.log2(a)
        X = torch.floor(lg) - 8 if case["rule"] == "floor" else torch.ceil(torch.log2(a / 448))
        X = torch.where(a > 0, X, -127.0).clamp(-127, 127)
        out["q"] = torch.clamp(b / torch.pow(2.0, X)[:, :, None], -448, 448).reshape(f.shape)
        sc = torch.pow(2.0, X)
        if case["layout"] == "k4":   # bytes behind the last block are 0: 2^-127
            sc = torch.nn.functional.pad(sc, (0, -sc.shape[1] % 4), value=2.0 ** -127)
            sc = sc.reshape(case["rows"], -1, 4).transpose(0, 1).contiguous()
        out["scale"] = sc
        return out
    if case["op"] == "norm_backward":
        s, dh, r = st["s"].to(D), st["dh"].to(D), st["rstd"].to(D)[:, None]
        g = dh * (1.0 if st["gamma"] is None else st["gamma"].to(D))
        dx = r * g - s * r ** 3 / case["cols"] * (g * s).sum(1, keepdim=True)
        if case["dsum"]:
            dx += st["dsum"].to(D)
        return {"dx": dx, "dgamma": (dh * s * r).sum(0)}

    T, E, k = case["tokens"], case["experts"], case["topk"]
    z = st["logits"].to(D)
    alive = z > -math.inf
    if case["score"] == "softmax":
        lse = torch.logsumexp(z, 1, keepdim=True)
        score = torch.where(alive, torch.exp(z - torch.where(lse > -math.inf, lse, 0.0)), 0.0)
        share = score
    else:
        score = torch.where(alive, 1 / (1 + torch.exp(-z)), 0.0)
        share = score / torch.where(alive.any(1, keepdim=True), score.sum(1, keepdim=True), 1.0)
    here = torch.ones(T, dtype=torch.bool, device=DEV) if st["mask"] is None else st["mask"].bool()
    out = {}
    ids = st.get("ids")
    if case["op"] in ("gate", "gate_balance"):
        key = z if st["bias"] is None else score + st["bias"].to(D)
        key = torch.where(alive & here[:, None], key, -math.inf)
        order = torch.argsort(key, dim=1, descending=True, stable=True)[:, :k]
        ids = torch.where(torch.take_along_dim(key, order, 1) > -math.inf, order, -1)
        w = torch.where(ids >= 0, torch.take_along_dim(score, ids.clamp(min=0).long(), 1), 0.0)
        if case["renorm"]:
            w = w / torch.where(w.sum(1, keepdim=True) > 0, w.sum(1, keepdim=True), 1.0)
        out = {"ids": ids.to(torch.int32), "weights": w * case["scale"]}
        if case["op"] == "gate":
            return out
    ids = ids.long()
    pick = torch.zeros(T, E + 1, dtype=D, device=DEV).scatter_(1, torch.where(ids >= 0, ids, E), 1.0)[:, :E]
    S = case["seqs"]
    end = st["seq_offs"].long()
    begin = torch.nn.functional.pad(end[:-1], (1, 0))

    def sums(x):   # over each sequence's tokens that count: differences of running sums
        run_ = torch.nn.functional.pad(torch.cumsum(torch.where(here[:, None], x, 0.0), 0), (0, 0, 1, 0))
        return run_[end] - run_[begin]

    n = sums(torch.ones(T, 1, dtype=D, device=DEV)).clamp(min=1)
    if case["op"] != "gate_backward":
        counts = sums(pick)
        f = counts * E / (k * n)
        loss = COEF / S * (f * sums(share) / n).sum()
        return out | {"loss": loss.view(1), "counts": counts.round().to(torch.int32), "dprob": COEF / S * f / n}
    t = torch.arange(T, device=DEV)
    member = ((t >= begin[:, None]) & (t < end[:, None]) & here).to(D)      # [S, T]
    dshare = (member.T @ st["dprob"].to(D)) * st["dloss"].to(D)
    dscore = dshare
    if case["score"] == "sigmoid":
        total = torch.where(alive.any(1, keepdim=True), score.sum(1, keepdim=True), 1.0)
        dscore = (dshare - (dshare * share).sum(1, keepdim=True)) / total
    if case["gate"]:
        dw = torch.zeros(T, E + 1, dtype=D, device=DEV).scatter_(1, torch.where(ids >= 0, ids, E), st["dweights"].to(D))[:, :E]
        dw *= case["scale"] * pick
        if case["renorm"]:
            chosen = (score * pick).sum(1, keepdim=True)
            chosen = torch.where(chosen > 0, chosen, 1.0)
            dw = pick * (dw / chosen - (dw * score).sum(1, keepdim=True) / chosen ** 2)
        dscore = dscore + dw
    if case["score"] == "sigmoid":
        dz = dscore * score * (1 - score)
    else:
        dz = score * (dscore - (dscore * score).sum(1, keepdim=True))
    return {"dlogits": torch.where(here[:, None], dz, 0.0)}
