"""Timed cases of the expert block's further forms: the linear layer in 8-bit integers, the whole expert block for a few
tokens, and the SwiGLU whose input is kept for the backward pass in 8 bits.

``run`` computes a case in plain torch operations, or, with ``own`` set, through the package's entry points; ``exact`` gives
the same outputs from the definitions in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
F8 = {"e4m3fn": (torch.float8_e4m3fn, 448.0), "e4m3fnuz": (torch.float8_e4m3fnuz, 240.0)}

MOST_LINEAR = 8192 * 4096 * 14336    # products of the largest linear layer
MOST_WEIGHTS = 32 * 4096 * 7168      # W1 elements of the largest expert block
MOST_SAVE = 16384 * 8192             # hidden elements of the largest SwiGLU


# ---------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # serving: one step of 16 sequences through a Llama3-8B linear layer
        dict(name="int8_decode", op="int8", rows=16, cols=4096, out=14336, experts=1, pad=0, f32=False),
        # a prompt's tokens through the same layer
        dict(name="int8_llama3_8b", op="int8", rows=8192, cols=4096, out=14336, experts=1, pad=0, f32=False),
        # DeepSeek-MoE-16B's first expert product, 8192 tokens of six experts each
        dict(name="int8_16b", op="int8", rows=49152, cols=2048, out=2816, experts=64, pad=0, f32=False),
        # odd sizes: a slice of wider rows, unaligned output rows, some experts without a row, fp32 output
        dict(name="int8_odd", op="int8", rows=509, cols=2064, out=1999, experts=11, pad=24, f32=True),
        # serving: a single token of DeepSeek-MoE-16B
        dict(name="few_one_16b", op="few", tokens=1, topk=6, experts=64, cols=2048, ffn=1408, fmt="fp8", local=False),
        # eight sequences of Llama4-Scout's MXFP8 experts
        dict(name="few_scout_mx", op="few", tokens=8, topk=1, experts=16, cols=5120, ffn=8192, fmt="mx_k4", local=False),
        # one GPU's share of DeepSeek-V3's experts: most of the 64 tokens' choices live elsewhere
        dict(name="few_v3_share", op="few", tokens=64, topk=8, experts=32, cols=7168, ffn=2048, fmt="fp8", local=True),
        # odd sizes, integer weights
        dict(name="few_odd", op="few", tokens=5, topk=3, experts=7, cols=1040, ffn=336, fmt="int8", local=True),
        # DeepSeek-MoE-16B's routed rows: the forward that keeps 8 bits
        dict(name="save_16b", op="save", rows=49152, ffn=1408, codec="e4m3fn", rule="floor", pad=0, a2=False),
        # and the backward that reads them, rowwise recipe
        dict(name="saved_bwd_16b", op="saved_backward", rows=49152, ffn=1408, codec="e4m3fn", rule="floor", a2=True),
        # Llama4-Scout's backward in the MXFP8 recipe, both forms
        dict(name="saved_bwd_scout_mx", op="saved_backward_mx", rows=16384, ffn=8192, experts=16, rule="floor", layout="k4"),
        # a short micro-batch, odd sizes, the fnuz codec
        dict(name="save_odd", op="save", rows=509, ffn=1056, codec="e4m3fnuz", rule="ceil", pad=40, a2=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["int8", "int8", "few", "few", "few", "save", "saved_backward", "saved_backward_mx"])
    if op == "int8":
        cols, out = 16 * _log_int(rng, 4, 512), _log_int(rng, 16, 16384)
        experts = rng.choice([1, 1, _log_int(rng, 2, 64)])
        experts = max(1, min(experts, 400_000_000 // (cols * out)))
        rows = _log_int(rng, 1, max(1, min(49152, MOST_LINEAR // (2 * cols * out), 3_000_000_000 // (4 * max(cols, out)))))
        return dict(op=op, rows=rows, cols=cols, out=out, experts=experts, pad=rng.choice([0, 8, 40]), f32=rng.random() < 0.3)
    if op == "few":
        fmt = rng.choice(["fp8", "fp8", "int8", "mx", "mx_k4"])
        step = 32 if fmt.startswith("mx") else 16
        cols, ffn = step * _log_int(rng, 256 // step, 7168 // step), step * _log_int(rng, 64 // step, 8192 // step)
        experts = max(1, min(_log_int(rng, 1, 64), MOST_WEIGHTS // (2 * ffn * cols)))
        return dict(op=op, tokens=_log_int(rng, 1, 64), topk=rng.randint(1, min(experts, 8)), experts=experts, cols=cols,
                    ffn=ffn, fmt=fmt, local=rng.random() < 0.3)
    if op == "saved_backward_mx":
        ffn = 128 * _log_int(rng, 1, 64)
        rows = _log_int(rng, 1, min(49152, MOST_SAVE // ffn))
        return dict(op=op, rows=rows, ffn=ffn, experts=_log_int(rng, 1, 64), rule=rng.choice(["floor", "ceil"]),
                    layout=rng.choice(["rows", "k4"]))
    ffn = 32 * _log_int(rng, 1, 448)
    case = dict(op=op, rows=_log_int(rng, 1, min(49152, MOST_SAVE // ffn)), ffn=ffn, codec=rng.choice(["e4m3fn", "e4m3fnuz"]),
                rule=rng.choice(["floor", "ceil"]), a2=rng.random() < 0.6)
    return dict(case, pad=rng.choice([0, 8, 40])) if op == "save" else case


def work(case):
    if case["op"] == "int8":
        M, K, N, E = case["rows"], case["cols"], case["out"], case["experts"]
        return {"bytes": 2 * M * K + min(E, M) * N * (K + 4) + M * N * (4 if case["f32"] else 2), "flops": 2 * M * N * K}
    if case["op"] == "few":
        T, E, K, F = case["tokens"], case["experts"], case["cols"], case["ffn"]
        k = case["topk"] * (0.25 if case["local"] else 1.0)          # choices of a token that live here
        used = E * (1 - (1 - min(1.0, k / E)) ** T)                  # experts that any token chose, on average
        scales = 3 * F * K / 32 if case["fmt"].startswith("mx") else 4 * (2 * F + K)
        return {"bytes": used * (3 * F * K + scales) + 4 * T * K + 8 * T * case["topk"], "flops": 6 * T * k * F * K}
    n = case["rows"] * case["ffn"]
    if case["op"] == "save":
        return {"bytes": n * (7 + 2 / 32 + (2 if case["a2"] else 0)) + 4 * case["rows"], "flops": 20 * n}
    if case["op"] == "saved_backward":
        return {"bytes": n * (10 + 2 / 32 + (2 if case["a2"] else 0)) + 4 * case["rows"], "flops": 30 * n}
    return {"bytes": n * (8 + 6 / 32), "flops": 30 * n}


# ---------------------------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _rows(g, rows, cols, pad=0):
    """bf16 activations with 1% outliers, a slice of rows `pad` elements wider."""
    x = torch.randn(rows, cols + pad, generator=g, device=DEV)
    x = torch.where(torch.rand(rows, cols + pad, generator=g, device=DEV) < 0.01, x * 30, x)
    return x.to(torch.bfloat16)[:, :cols]


def _offs(g, rows, experts):
    """Inclusive ends of the experts' rows: experts of unequal popularity, every row in a group; and the largest group."""
    p = 0.3 + torch.rand(experts, generator=g, device=DEV)
    counts = torch.bincount(torch.multinomial(p, rows, replacement=True, generator=g), minlength=experts)
    return counts.cumsum(0).to(torch.int32), int(counts.max())


def _weights(g, rows, cols, fmt):
    """Quantized weights of N(0, 0.02): codes [rows, cols] and their scales."""
    w = torch.randn(rows, cols, generator=g, device=DEV).mul_(0.02).to(torch.bfloat16).float()
    if fmt.startswith("mx"):
        q, X = _mx(w, "floor")
        code = (X + 127).to(torch.uint8)
        return q, _k4(code) if fmt == "mx_k4" else code
    fmax = 127.0 if fmt == "int8" else 448.0
    s = fmax / w.abs().amax(1).clamp(min=1e-12)
    w *= s[:, None]
    return (w.round_().to(torch.int8) if fmt == "int8" else w.clamp_(-fmax, fmax).to(torch.float8_e4m3fn)), s


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=case)
    if case["op"] == "int8":
        s["x"] = _rows(g, case["rows"], case["cols"], case["pad"])
        E, N = case["experts"], case["out"]
        q, sc = _weights(g, E * N, case["cols"], "int8")
        s["w"], s["ws"] = q.view(E, N, -1), sc.view(E, N)
        s["offs"], s["most"] = _offs(g, case["rows"], E)
        return s
    if case["op"] == "few":
        T, E, k, K, F = case["tokens"], case["experts"], case["topk"], case["cols"], case["ffn"]
        s["x"] = _rows(g, T, K)
        logits = torch.randn(T, E, generator=g, device=DEV) + 0.5 * torch.randn(E, generator=g, device=DEV)
        top = torch.topk(logits, k, dim=1)
        s["weights"], s["ids"] = torch.softmax(top.values, 1), top.indices.to(torch.int32)
        if case["local"]:   # three of four choices live on other GPUs
            s["ids"] = torch.where(torch.rand(T, k, generator=g, device=DEV) < 0.25, s["ids"], -1)
        s["w1"], s["s1"] = _weights(g, E * 2 * F, K, case["fmt"])
        s["w2"], s["s2"] = _weights(g, E * K, F, case["fmt"])
        s["w1"], s["w2"] = s["w1"].view(E, 2 * F, K), s["w2"].view(E, K, F)
        return s
    h1 = _rows(g, case["rows"], 2 * case["ffn"], case.get("pad", 0))
    if case["op"] == "save":
        s["h1"] = h1
        return s
    s["hq"], X = _mx(h1.float(), case["rule"])
    s["hs"] = (X + 127).to(torch.uint8)
    s["da2"] = (1e-3 * torch.randn(case["rows"], case["ffn"], generator=g, device=DEV)).to(torch.bfloat16)
    if case["op"] == "saved_backward_mx":
        s["offs"], _ = _offs(g, case["rows"], case["experts"])
    return s


# ---------------------------------------------------------------------------------------------- plain forms

def _mx_exponent(amax, rule):
    """floor(log2 amax) - 8, one more under the CEIL rule where the significand is over 1.75; -127 for a zero block."""
    m, e = torch.frexp(amax)                       # amax = m 2^e, m in [0.5, 1)
    X = e - 9 + ((m > 0.875).to(e.dtype) if rule == "ceil" else 0)
    return torch.where(amax == 0, -127, X.clamp(-127, 127))


def _mx(f, rule):
    """e4m3 codes of f in blocks of 32 along the last dimension, and the blocks' exponents."""
    b = f.reshape(*f.shape[:-1], -1, 32)
    X = _mx_exponent(b.abs().amax(-1), rule)
    q = (b * torch.exp2(-X.float())[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return q.view(f.shape), X


def _k4(code):
    """Row-major scale bytes [R, NB] as [ceil(NB / 4), R, 4]."""
    R, NB = code.shape
    p = torch.zeros(R, -(-NB // 4) * 4, dtype=torch.uint8, device=code.device)
    p[:, :NB] = code
    return p.view(R, -1, 4).permute(1, 0, 2).contiguous()


def _rowwise(f, codec):
    dt, fmax = F8[codec]
    scale = fmax / f.abs().amax(1).clamp(min=1e-12)
    return (f * scale[:, None]).clamp(-fmax, fmax).to(dt), scale


def _from_k4(p, rows, nb):
    return p.view(-1, rows, 4).permute(1, 0, 2).reshape(rows, -1)[:, :nb]


def _groups(offs, rows):
    """Each row's group, and the groups' first rows."""
    of = torch.searchsorted(offs.long(), torch.arange(rows, device=offs.device), right=True)
    return of, torch.nn.functional.pad(offs.long()[:-1], (1, 0))


def _plain_int8(st):
    case, x = st["case"], st["x"].float()
    M, E = case["rows"], case["experts"]
    s = 127.0 / x.abs().amax(1).clamp(min=1e-12)
    q = (x * s[:, None]).clamp(-127, 127).round()
    if E == 1:
        y = (q @ st["w"][0].float().t()) / st["ws"][0]
    else:   # a batched product over the experts' rows, padded to the largest group
        of, first = _groups(st["offs"], M)
        at = torch.arange(M, device=DEV) - first[of]
        rows = q.new_zeros(E, st["most"], case["cols"])
        rows[of, at] = q
        y = torch.bmm(rows, st["w"].float().transpose(1, 2).contiguous())[of, at] / st["ws"][of]
    y = y / s[:, None]
    return {"y": y if case["f32"] else y.to(torch.bfloat16)}


def _decoded(case, q, s, at, rows_each):
    """Experts `at` (all with None) of quantized weights q [E, rows_each, cols] in 32 bits."""
    if case["fmt"].startswith("mx"):
        nb = q.shape[2] // 32
        code = _from_k4(s, q.shape[0] * rows_each, nb) if case["fmt"] == "mx_k4" else s
        code = code.reshape(-1, rows_each, nb)
        if at is not None:
            q, code = q.view(torch.uint8)[at].view(q.dtype), code[at]
        f = torch.exp2(code.float() - 127)
        return (q.float().view(*q.shape[:2], nb, 32) * f[..., None]).view(q.shape)
    s = s.view(-1, rows_each)
    if at is not None:
        q, s = q.view(torch.uint8)[at].view(q.dtype), s[at]
    return q.float() / s[..., None]


def _plain_few(st):
    case, ids = st["case"], st["ids"].long()
    T, k = ids.shape
    E, K, F = case["experts"], case["cols"], case["ffn"]
    here, e = (ids >= 0).view(-1), ids.clamp(min=0).view(-1)
    x = st["x"].float()
    if T * k <= E:   # few choices: their experts' weights; else every expert's
        h = torch.bmm(_decoded(case, st["w1"], st["s1"], e, 2 * F), x.repeat_interleave(k, 0)[:, :, None])[:, :, 0]
    else:
        w = _decoded(case, st["w1"], st["s1"], None, 2 * F)
        h = (x @ w.view(E * 2 * F, K).t()).view(T, E, 2 * F)[torch.arange(T * k, device=DEV) // k, e]
    g, u = h[:, :F], h[:, F:]
    a = (g * torch.sigmoid(g) * u).to(torch.bfloat16).float()
    if T * k <= E:
        o = torch.bmm(_decoded(case, st["w2"], st["s2"], e, K), a[:, :, None])[:, :, 0]
    else:
        w = _decoded(case, st["w2"], st["s2"], None, K)
        o = (a @ w.view(E * K, F).t()).view(T * k, E, K)[torch.arange(T * k, device=DEV), e]
    o = torch.where(here[:, None], o * st["weights"].view(-1, 1), 0.0)
    return {"y": o.view(T, k, K).sum(1).to(torch.bfloat16)}


def _plain_save(st):
    case, h1 = st["case"], st["h1"].float()
    g, u = h1[:, :case["ffn"]], h1[:, case["ffn"]:]
    a = g * torch.sigmoid(g) * u
    out = {}
    out["q"], out["scale"] = _rowwise(a, case["codec"])
    out["hq"], X = _mx(h1, case["rule"])
    out["hs"] = (X + 127).to(torch.uint8).view(torch.float8_e8m0fnu)
    if case["a2"]:
        out["a2"] = a.to(torch.bfloat16)
    return out


def _plain_gradient(st):
    """SwiGLU's input gradient and its output from the kept codes, in 32 bits."""
    F = st["case"]["ffn"]
    h = st["hq"].float().view(-1, 2 * F // 32, 32) * torch.exp2(st["hs"].float() - 127)[:, :, None]
    h = h.view(-1, 2 * F)
    g, u, d = h[:, :F], h[:, F:], st["da2"].float()
    s = torch.sigmoid(g)
    return torch.cat([d * u * s * (1 + g * (1 - s)), d * g * s], 1), g * s * u


def _plain_saved_backward(st):
    case = st["case"]
    dh, a = _plain_gradient(st)
    out = {"dh1": dh.to(torch.bfloat16)}
    out["q"], out["scale"] = _rowwise(dh, case["codec"])
    if case["a2"]:
        out["a2"] = a.to(torch.bfloat16)
    return out


def _padded(st, x):
    """Rows of x moved to groups padded to whole blocks of 32 rows, transposed; and the padded ends."""
    M, E = st["case"]["rows"], st["case"]["experts"]
    of, first = _groups(st["offs"], M)
    counts = st["offs"].long() - first
    ends = ((counts + 31) // 32 * 32).cumsum(0)
    to = torch.arange(M, device=DEV) - first[of] + torch.nn.functional.pad(ends[:-1], (1, 0))[of]
    p = x.new_zeros((M + 31 * E + 31) // 32 * 32, x.shape[1])
    p[to] = x
    return p.t().contiguous(), ends.to(torch.int32)


def _scales(X, layout):
    code = (X + 127).to(torch.uint8)
    return (_k4(code) if layout == "k4" else code).view(torch.float8_e8m0fnu)


def _plain_saved_backward_mx(st):
    case = st["case"]
    dh = _plain_gradient(st)[0].to(torch.bfloat16).float()   # the codes are those of the bf16 gradient
    out = {}
    out["q"], X = _mx(dh, case["rule"])
    out["scale"] = _scales(X, case["layout"])
    t, out["offs_pad"] = _padded(st, dh)
    out["q_t"], X = _mx(t, case["rule"])
    out["scale_t"] = _scales(X, case["layout"])
    return out


# ---------------------------------------------------------------------------------------------- one pass

def run(st):
    if own:
        return _own(st)
    op = st["case"]["op"]
    if op == "int8":
        return _plain_int8(st)
    if op == "few":
        return _plain_few(st)
    if op == "save":
        return _plain_save(st)
    return _plain_saved_backward(st) if op == "saved_backward" else _plain_saved_backward_mx(st)


def _own(st):
    import mxfp8_quantized_moe_amd as fm
    case, op = st["case"], st["case"]["op"]
    if op == "int8":
        q, s = fm.quantize_rowwise(st["x"], codec=fm.INT8)
        return {"y": fm.grouped_mm_scaled(fm.GROUPED_M, q, fm.OPD_INT8, s, st["w"], fm.OPD_INT8, st["ws"], fm.SCALE_F32,
                                          st["offs"], case["experts"], case["rows"], case["out"], case["cols"],
                                          out_dtype=fm.OUT_F32 if case["f32"] else fm.OUT_BF16)}
    if op == "few":
        kind = {"mx": fm.SCALE_E8M0, "mx_k4": fm.SCALE_E8M0_K4}.get(case["fmt"], fm.SCALE_F32)
        return {"y": fm.moe_few_tokens(st["x"], st["ids"], st["weights"], st["w1"], st["s1"], st["w2"], st["s2"],
                                       w_fmt=fm.OPD_INT8 if case["fmt"] == "int8" else fm.OPD_E4M3FN, scale_kind=kind)}
    rule = fm.MX_CEIL if case["rule"] == "ceil" else fm.MX_FLOOR_OCP
    if op == "saved_backward_mx":
        _, q, s, q_t, s_t, offs_pad = fm.swiglu_backward_quantize_mx_dual_saved(
            st["da2"], st["hq"], st["hs"], st["offs"], rule=rule,
            layout=fm.MX_LAYOUT_K4 if case["layout"] == "k4" else fm.MX_LAYOUT_ROWS)
        e4, e8 = torch.float8_e4m3fn, torch.float8_e8m0fnu
        return {"q": q.view(e4), "scale": s.view(e8), "offs_pad": offs_pad, "q_t": q_t.view(e4), "scale_t": s_t.view(e8)}
    dt, codec = F8[case["codec"]][0], fm.E4M3FN if case["codec"] == "e4m3fn" else fm.E4M3FNUZ
    if op == "save":
        a2, q, scale, hq, hs = fm.swiglu_quantize_rowwise_save(st["h1"], codec=codec, rule=rule, keep_bf16=case["a2"])
        out = {"q": q.view(dt), "scale": scale, "hq": hq.view(torch.float8_e4m3fn), "hs": hs.view(torch.float8_e8m0fnu)}
    else:
        dh1, q, scale, a2 = fm.swiglu_backward_quantize_rowwise_saved(st["da2"], st["hq"], st["hs"], codec=codec,
                                                                      want_a2=case["a2"])
        out = {"dh1": dh1, "q": q.view(dt), "scale": scale}
    return out | {"a2": a2} if case["a2"] else out


# ---------------------------------------------------------------------------------------------- definitions in 64 bits

def _exact_int8(case, st):
    D = torch.float64
    # the codes are whole numbers that fp32 decides: fp32(127 / max), fp32(x s), ties to even
    x = st["x"].float()
    s = 127.0 / torch.maximum(x.abs().max(1).values, torch.tensor(1e-12, device=DEV))
    q = torch.round(torch.einsum("rc,r->rc", x, s)).clamp(-127, 127).to(D)
    y = torch.empty(case["rows"], case["out"], dtype=D, device=DEV)
    begin = 0
    for e, end in enumerate(st["offs"].tolist()):
        y[begin:end] = torch.mm(q[begin:end], st["w"][e].to(D).t().contiguous()) * (1 / st["ws"][e].to(D))
        begin = end
    return {"y": y * (1 / s.to(D))[:, None]}


def _exact_few(case, st):
    D = torch.float64
    E, K, F, T = case["experts"], case["cols"], case["ffn"], case["tokens"]
    x, ids, w = st["x"].to(D), st["ids"].long(), st["weights"].to(D)
    y = torch.zeros(T, K, dtype=D, device=DEV)

    def expert(q, s, e, n):
        v = q[e].to(D)
        if not case["fmt"].startswith("mx"):
            return v * (1 / s.view(E, n)[e].to(D))[:, None]
        nb = v.shape[1] // 32
        if case["fmt"] == "mx_k4":
            code = s[:, e * n:(e + 1) * n, :].transpose(0, 1).reshape(n, -1)[:, :nb]
        else:
            code = s.view(E, n, nb)[e]
        return v * torch.pow(2.0, code.to(D) - 127).repeat_interleave(32, 1)

    for e in range(E):
        h = x @ expert(st["w1"], st["s1"], e, 2 * F).t()
        a = h[:, :F] / (1 + torch.exp(-h[:, :F])) * h[:, F:]
        o = a @ expert(st["w2"], st["s2"], e, K).t()
        y += torch.where(ids == e, w, 0.0).sum(1, keepdim=True) * o
    return {"y": y}


def _exact_mx(v, rule):
    """Scaled values (not yet rounded to codes) and scales of blocks of 32 along the last dimension."""
    b = v.reshape(v.shape[0], -1, 32)
    a = b.abs().max(2).values
    X = torch.floor(torch.log2(a)) - 8 if rule == "floor" else torch.ceil(torch.log2(a / 448))
    X = torch.where(a > 0, X, -127.0).clamp(-127, 127)
    return torch.clamp(b / torch.pow(2.0, X)[:, :, None], -448, 448).reshape(v.shape), torch.pow(2.0, X)


def _exact_k4(sc):
    sc = torch.nn.functional.pad(sc, (0, -sc.shape[1] % 4), value=2.0 ** -127)   # bytes behind the last block are 0
    return sc.reshape(sc.shape[0], -1, 4).transpose(0, 1).contiguous()


def exact(case, seed):
    st = prepare(case, seed)
    D = torch.float64
    if case["op"] == "int8":
        return _exact_int8(case, st)
    if case["op"] == "few":
        return _exact_few(case, st)
    F = case["ffn"]
    if case["op"] == "save":
        h = st["h1"].to(D)
        a = h[:, :F] / (1 + torch.exp(-h[:, :F])) * h[:, F:]
        scale = F8[case["codec"]][1] / a.abs().max(1).values.clamp(min=1e-12)
        out = {"q": a * scale[:, None], "scale": scale}
        out["hq"], out["hs"] = _exact_mx(h, case["rule"])
        return out | {"a2": a} if case["a2"] else out
    h = st["hq"].to(D) * torch.pow(2.0, st["hs"].to(D) - 127).repeat_interleave(32, 1)
    g, u, d = h[:, :F], h[:, F:], st["da2"].to(D)
    p, n = 1 / (1 + torch.exp(-g)), 1 / (1 + torch.exp(g))
    dh = torch.cat([d * u * (p + g * p * n), d * g * p], 1)
    if case["op"] == "saved_backward":
        scale = F8[case["codec"]][1] / dh.abs().max(1).values.clamp(min=1e-12)
        out = {"dh1": dh, "q": dh * scale[:, None], "scale": scale}
        return out | {"a2": g * p * u} if case["a2"] else out
    dh = dh.to(torch.bfloat16).to(D)
    M, E = case["rows"], case["experts"]
    pad = torch.zeros(2 * F, (M + 31 * E + 31) // 32 * 32, dtype=D, device=DEV)
    ends, begin, at = [], 0, 0
    for end in st["offs"].tolist():
        pad[:, at:at + end - begin] = dh[begin:end].t()
        at += -(-(end - begin) // 32) * 32
        ends.append(at)
        begin = end
    out = {"offs_pad": torch.tensor(ends, dtype=torch.int32, device=DEV)}
    out["q"], sc = _exact_mx(dh, case["rule"])
    out["q_t"], sc_t = _exact_mx(pad, case["rule"])
    k4 = case["layout"] == "k4"
    return out | {"scale": _exact_k4(sc) if k4 else sc, "scale_t": _exact_k4(sc_t) if k4 else sc_t}
