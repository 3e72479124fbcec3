"""The SwiGLU with its input kept in 8 bits at the C ABI and in the binding: every refusal (no GPU)."""
import pytest
import torch

import mxfp8_quantized_moe_amd as fm
from mxfp8_quantized_moe_amd import _lib as L

P = 0x10000


@pytest.fixture(scope="module")
def lib():
    return L.lib()


def refused(f, ok, **kw):
    a = dict(ok, **kw)
    return f(*[a[k] for k in ok], None)


def test_save(lib):
    f = lib.swiglu_quantize_rowwise_save
    ok = dict(h1=P, rows=4, F=64, ld=128, codec=0, rule=0, a2=P, q=P, scale=P, hq=P, hs=P)
    for k in ("h1", "q", "scale", "hq", "hs"):
        assert refused(f, ok, **{k: None}) == L.ERR_NULL, k
    for k in ("h1", "a2", "q", "hq"):
        assert refused(f, ok, **{k: P + 8}) == L.ERR_ALIGN, k
    assert refused(f, ok, scale=P + 2) == L.ERR_ALIGN
    for kw in (dict(codec=2), dict(codec=L.INT8), dict(rule=2)):
        assert refused(f, ok, **kw) == L.ERR_ENUM
    for kw in (dict(rows=-1), dict(F=-32), dict(ld=120), dict(F=1 << 40, ld=1 << 42), dict(rows=1 << 24)):
        assert refused(f, ok, **kw) == L.ERR_SHAPE
    for kw in (dict(F=48), dict(ld=132)):
        assert refused(f, ok, **kw) == L.ERR_ALIGN
    assert refused(f, dict(ok, h1=None, q=None, scale=None, hq=None, hs=None, a2=None), rows=0) == L.OK


def test_saved_backward(lib):
    f = lib.swiglu_backward_quantize_rowwise_saved
    ok = dict(da2=P, hq=P, hs=P, rows=4, F=64, codec=0, dh1=P, q=P, scale=P, a2=P)
    for k in ("da2", "hq", "hs", "q", "scale"):
        assert refused(f, ok, **{k: None}) == L.ERR_NULL, k
    assert refused(f, ok, dh1=None, q=None, scale=None, a2=None) == L.ERR_NULL      # nothing asked for
    for k in ("da2", "hq", "dh1", "q", "a2"):
        assert refused(f, ok, **{k: P + 8}) == L.ERR_ALIGN, k
    assert refused(f, ok, scale=P + 2) == L.ERR_ALIGN
    assert refused(f, ok, F=48) == L.ERR_ALIGN
    for kw in (dict(codec=3), dict(codec=L.INT8)):
        assert refused(f, ok, **kw) == L.ERR_ENUM
    for kw in (dict(rows=-1), dict(F=-32), dict(rows=1 << 24), dict(F=1 << 40)):
        assert refused(f, ok, **kw) == L.ERR_SHAPE


@pytest.mark.parametrize("bwd", [False, True])
def test_mx_dual_saved(lib, bwd):
    f = lib.swiglu_backward_quantize_mx_dual_saved if bwd else lib.swiglu_quantize_mx_dual_saved
    ok = dict(hq=P, hs=P, rows=64, F=128, offs=P, E=4, rule=0, layout=1, out=None, q=P, sc=P, q_t=P, sc_t=P, rows_pad=192, offs_pad=P)
    if bwd:
        ok = dict(da2=P, **ok)
    for k in ["hq", "hs", "offs", "q", "sc", "q_t", "sc_t"]:
        assert refused(f, ok, **{k: None}) == L.ERR_NULL, k
    assert refused(f, ok, rule=2) == L.ERR_ENUM
    assert refused(f, ok, layout=2) == L.ERR_ENUM
    for kw in (dict(rows=-1), dict(F=-128), dict(E=0), dict(rows_pad=160), dict(F=1 << 40)):
        assert refused(f, ok, **kw) == L.ERR_SHAPE, kw
    assert refused(f, ok, F=48) == L.ERR_ALIGN
    assert refused(f, ok, rows_pad=200) == L.ERR_ALIGN
    for k in ["hq", "q", "q_t", "out"] + (["da2"] if bwd else []):
        assert refused(f, ok, **{k: P + 8}) == L.ERR_ALIGN, k
    if bwd:
        assert refused(f, ok, F=96) == L.ERR_ALIGN


def test_binding_refuses():
    h1 = torch.zeros(4, 128, dtype=torch.bfloat16)
    for bad in (h1.float(), h1[0], h1[:, :96], h1.t(), torch.zeros(4, 96, dtype=torch.bfloat16)):
        with pytest.raises(ValueError, match="swiglu_quantize_rowwise_save"):
            fm.swiglu_quantize_rowwise_save(bad)
    with pytest.raises(ValueError, match="GPU tensors"):
        fm.swiglu_quantize_rowwise_save(h1)
    da, hq, hs = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(4, 128, dtype=torch.uint8), torch.zeros(4, 4, dtype=torch.uint8)
    offs = torch.zeros(2, dtype=torch.int32)
    bad = [dict(da2=da.float()), dict(da2=da[:3]), dict(da2=da[:, ::2]), dict(hq=hq.float()), dict(hq=hq[:, :96]),
           dict(hq=torch.zeros(4, 136, dtype=torch.uint8)[:, :128]), dict(hs=hs.int()), dict(hs=hs[:, :2]), dict(hs=hs.t())]
    for kw in bad:
        with pytest.raises(ValueError, match="rowwise_saved"):
            fm.swiglu_backward_quantize_rowwise_saved(**dict(dict(da2=da, hq=hq, hs=hs), **kw))
        with pytest.raises(ValueError, match="mx_dual_saved"):
            fm.swiglu_backward_quantize_mx_dual_saved(**dict(dict(da2=da, hq=hq, hs=hs, offs=offs), **kw))
    with pytest.raises(ValueError, match="no result"):
        fm.swiglu_backward_quantize_rowwise_saved(da, hq, hs, keep_bf16=False, codes=False)
    for kw in (dict(offs=offs.long()), dict(offs=offs[:0])):
        with pytest.raises(ValueError, match="offs"):
            fm.swiglu_quantize_mx_dual_saved(**dict(dict(hq=hq, hs=hs, offs=offs), **kw))
