"""moe_few_tokens at the C ABI and in the binding: every refusal (no GPU)."""
import pytest
import torch

import mxfp8_quantized_moe_amd as fm
from mxfp8_quantized_moe_amd import _lib as L

P = 0x10000


@pytest.fixture(scope="module")
def lib():
    return L.lib()


OK = dict(x=P, T=4, K=64, ld=64, ids=P, w=P, topk=2, w1=P, s1=P, w2=P, s2=P, fmt=0, sk=0, E=8, F=32, y=P, ws=P)


def call(lib, **kw):
    a = dict(OK, **kw)
    return lib.moe_few_tokens(*[a[k] for k in OK], None)


def test_refusals(lib):
    for k in ("x", "ids", "w", "w1", "s1", "w2", "s2", "y", "ws"):
        assert call(lib, **{k: None}) == L.ERR_NULL, k
        assert call(lib, **{k: P + 2}) == L.ERR_ALIGN, k
    assert call(lib, fmt=3) == L.ERR_ENUM
    assert call(lib, sk=4) == L.ERR_ENUM
    for kw in (dict(T=-1), dict(K=-16), dict(F=-16), dict(topk=0), dict(E=0), dict(ld=56), dict(K=1 << 40, ld=1 << 40),
               dict(F=1 << 40), dict(F=(1 << 17) + 32), dict(K=(1 << 17) + 32, ld=1 << 18), dict(ld=(1 << 24) + 8)):
        assert call(lib, **kw) == L.ERR_SHAPE, kw
    for kw in (dict(fmt=1), dict(fmt=2), dict(fmt=4, sk=1), dict(fmt=4, sk=3), dict(sk=2), dict(T=65), dict(T=64, topk=17),
               dict(T=1, topk=1025), dict(E=1025)):
        assert call(lib, **kw) == L.ERR_UNSUPPORTED, kw
    for kw in (dict(K=72, ld=72), dict(F=24), dict(K=48, ld=48, sk=1), dict(F=48, sk=3), dict(ld=68)):
        assert call(lib, **kw) == L.ERR_ALIGN, kw
    assert call(lib, sk=1, s1=P + 1, w1=P + 1) == L.ERR_ALIGN   # e8m0 bytes may start anywhere, codes not


def test_nothing_to_do(lib):
    assert lib.moe_few_tokens(None, 0, 64, 64, None, None, 2, None, None, None, None, 0, 0, 8, 32, None, None, None) == L.OK
    assert lib.moe_few_tokens(None, 4, 0, 0, None, None, 2, None, None, None, None, 0, 0, 8, 32, None, None, None) == L.OK


def test_workspace_bytes():
    assert fm.moe_few_tokens_workspace_bytes(64, 16, 2048, 4096) >= 64 * 16 * (4096 * 2 + 2048 * 4)
    for bad in ((-1, 1, 16, 16), (65, 1, 16, 16), (64, 17, 16, 16), (4, 0, 16, 16), (4, 1, 16, -16), (4, 1, -16, 16), (4, 1, 1 << 21, 16), (4, 1, 16, (1 << 17) + 16)):
        assert fm.moe_few_tokens_workspace_bytes(*bad) == -1


def test_binding_refuses():
    x, ids, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    w1, s1 = torch.zeros(8, 64, 64, dtype=torch.uint8), torch.zeros(8, 64)
    w2, s2 = torch.zeros(8, 64, 32, dtype=torch.uint8), torch.zeros(8, 64)
    good = dict(x=x, ids=ids, weights=w, w1=w1, w1_scale=s1, w2=w2, w2_scale=s2)
    bad = [dict(x=x.float()), dict(x=x[:, ::2]), dict(x=x[0]), dict(ids=ids.long()), dict(ids=ids[:3]), dict(weights=w.double()),
           dict(weights=w[:, :1]), dict(w1=w1[:, :63]), dict(w1=w1.float()), dict(w1=w1.transpose(1, 2)), dict(w2=w2[:7]),
           dict(w2=w2[:, :, :16]), dict(w1_scale=s1.double()), dict(w2_scale=s2[:, :3]), dict(w_fmt=fm.OPD_INT8, w1=w1.view(torch.float8_e4m3fn)),
           dict(scale_kind=fm.SCALE_E8M0), dict(scale_kind=fm.SCALE_E8M0_K4)]
    for kw in bad:
        with pytest.raises(ValueError, match="moe_few_tokens"):
            fm.moe_few_tokens(**dict(good, **kw))
    with pytest.raises(ValueError, match="GPU tensors"):
        fm.moe_few_tokens(**good)
