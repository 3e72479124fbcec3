"""Refusals of the gate's and the balance loss's entry points, on the host: no HIP call is reached."""
import math

import pytest
import torch

import mxfp8_quantized_moe_amd as fm
from mxfp8_quantized_moe_amd import _lib as L

P, MIS = 0x10000, 0x10001


@pytest.fixture(scope="module")
def lib():
    return L.lib()


LOGITS = dict(logits=P, dt=1, T=4, E=8, ld=8, k=2, score=0)
GATE = dict(LOGITS, bias=P, mask=P, renorm=1, rs=1.0, ids=P, w=P)
LOSS = dict(seq=P, S=2, coef=0.1, loss=P, counts=P, dprob=P, ws=P, stream=None)
FORMS = {
    "moe_gate": dict(GATE, stream=None),
    "moe_gate_balance": dict(GATE, **LOSS),
    "moe_balance_loss": dict(LOGITS, mask=P, ids=P, **LOSS),
    "moe_gate_backward": dict(LOGITS, mask=P, renorm=0, rs=1.0, ids=P, dw=P, seq=P, S=2, dprob=P, dloss=P, dz=P, stream=None),
}


def refused(lib, name, **kw):
    a = dict(FORMS[name])
    assert set(kw) <= set(a)
    a.update(kw)
    return getattr(lib, name)(*a.values())


@pytest.mark.parametrize("name", FORMS)
def test_logits_rejections(lib, name):
    r = lambda **kw: refused(lib, name, **kw)  # noqa: E731
    assert r(dt=2) == L.ERR_ENUM
    assert r(score=2) == L.ERR_ENUM
    assert r(T=-1) == L.ERR_SHAPE
    assert r(E=0) == L.ERR_SHAPE
    assert r(ld=7) == L.ERR_SHAPE
    assert r(k=0) == L.ERR_SHAPE
    assert r(k=9) == L.ERR_SHAPE
    assert r(E=1025, ld=1025) == L.ERR_UNSUPPORTED
    assert r(E=128, ld=128, k=65) == L.ERR_UNSUPPORTED
    assert r(T=1 << 31) == L.ERR_SHAPE
    assert r(T=1 << 30, k=4) == L.ERR_SHAPE
    assert r(logits=None) == L.ERR_NULL
    assert r(logits=P + 2) == L.ERR_ALIGN
    assert r(logits=MIS, dt=0) == L.ERR_ALIGN


def test_gate_rejections(lib):
    for name in ("moe_gate", "moe_gate_balance"):
        for v in (math.inf, -math.inf, math.nan):
            assert refused(lib, name, rs=v) == L.ERR_VALUE
        for p in ("ids", "w"):
            assert refused(lib, name, **{p: None}) == L.ERR_NULL
        for p in ("bias", "ids", "w"):
            assert refused(lib, name, **{p: P + 2}) == L.ERR_ALIGN
    assert refused(lib, "moe_gate", T=0, logits=None, ids=None, w=None) == L.OK


def test_loss_rejections(lib):
    for name in ("moe_balance_loss", "moe_gate_balance"):
        assert refused(lib, name, S=0) == L.ERR_SHAPE
        assert refused(lib, name, S=(1 << 20) + 1) == L.ERR_SHAPE
        assert refused(lib, name, coef=math.nan) == L.ERR_VALUE
        assert refused(lib, name, seq=None) == L.ERR_NULL          # several sequences need their ends
        for p in ("ids", "loss", "counts", "dprob", "ws"):
            assert refused(lib, name, **{p: None}) == L.ERR_NULL, p
            assert refused(lib, name, **{p: P + 2}) == L.ERR_ALIGN, p
        assert refused(lib, name, seq=P + 2) == L.ERR_ALIGN
        assert refused(lib, name, ws=P + 8) == L.ERR_ALIGN
    assert lib.moe_balance_workspace_bytes(-1, 8, 1) == -1
    assert lib.moe_balance_workspace_bytes(8, 0, 1) == -1
    assert lib.moe_balance_workspace_bytes(8, 1025, 1) == -1
    assert lib.moe_balance_workspace_bytes(8, 8, 0) == -1
    assert lib.moe_balance_workspace_bytes(0, 8, 1) > 0


def test_backward_rejections(lib):
    r = lambda **kw: refused(lib, "moe_gate_backward", **kw)  # noqa: E731
    assert r(rs=math.nan) == L.ERR_VALUE
    assert r(S=0) == L.ERR_SHAPE
    assert r(seq=None) == L.ERR_NULL
    assert r(dw=None, dprob=None) == L.ERR_NULL                    # nothing to propagate
    assert r(ids=None) == L.ERR_NULL
    assert r(dz=None) == L.ERR_NULL
    for p in ("ids", "dw", "seq", "dprob", "dloss", "dz"):
        assert r(**{p: P + 2}) == L.ERR_ALIGN, p
    assert r(T=0, logits=None, ids=None, dw=None, dz=None) == L.OK


def test_binding_refusals():
    z, ids, dw = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    calls = {
        "gate": lambda **k: fm.moe_gate(**dict(dict(logits=z, topk=2), **k)),
        "both": lambda **k: fm.moe_gate_balance(**dict(dict(logits=z, topk=2, coef=0.1), **k)),
        "loss": lambda **k: fm.moe_balance_loss(**dict(dict(logits=z, ids=ids, coef=0.1), **k)),
        "back": lambda **k: fm.moe_gate_backward(**dict(dict(logits=z, ids=ids, dweights=dw), **k)),
        "lossback": lambda **k: fm.moe_balance_loss_backward(**dict(dict(logits=z, dprob=torch.zeros(1, 8)), **k)),
    }
    for name, call in calls.items():
        for bad in (z.double(), z[0], z.t(), z[:, ::2], z[:, :0], z[:1].expand(4, 8)):
            with pytest.raises(ValueError, match="logits"):
                call(logits=bad)
        for bad in (torch.ones(3, dtype=torch.uint8), torch.ones(4), torch.ones(8, dtype=torch.bool)[::2]):
            with pytest.raises(ValueError, match="token_mask"):
                call(token_mask=bad)
        with pytest.raises(ValueError, match="GPU"):
            call()
    for name in ("gate", "both"):
        for k in (0, -1, 9):
            with pytest.raises(ValueError, match="topk"):
                calls[name](topk=k)
        for bad in (torch.zeros(7), torch.zeros(8, dtype=torch.float64)):
            with pytest.raises(ValueError, match="bias"):
                calls[name](bias=bad)
    for name in ("both", "loss"):
        for bad in (torch.zeros(0, dtype=torch.int32), torch.zeros(2, dtype=torch.int64), torch.zeros(1, 2, dtype=torch.int32)):
            with pytest.raises(ValueError, match="seq_offs"):
                calls[name](seq_offs=bad)
    for name in ("loss", "back"):
        for bad in (ids.long(), ids[:3], ids.t().contiguous().t(), ids[:, 0]):
            with pytest.raises(ValueError, match="ids"):
                calls[name](ids=bad)
    for bad in (dw.double(), dw[:3], torch.zeros(4, 3), torch.zeros(9)):
        with pytest.raises(ValueError, match="dweights"):
            calls["back"](dweights=bad)
    with pytest.raises(ValueError, match="dprob"):
        calls["back"](dloss=torch.ones(1))
    with pytest.raises(ValueError, match="dprob"):
        calls["lossback"](dprob=None)
    for bad in (torch.zeros(2, 8), torch.zeros(8), torch.zeros(1, 8, dtype=torch.float64)):
        with pytest.raises(ValueError, match="dprob"):
            calls["lossback"](dprob=bad)
    with pytest.raises(ValueError, match="dloss"):
        calls["lossback"](dloss=torch.ones(2))


def test_more_experts_than_an_int32_counts():
    """2^32 + 5 experts are not taken for five."""
    z = torch.empty((0, 2**32 + 5), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="fewer than"):
        fm.moe_gate(z, 2)
