"""moe_few_tokens takes e8m0 scales as bytes or as torch's e8m0 type, as the kept SwiGLU does (no GPU)."""
import pytest
import torch

import mxfp8_quantized_moe_amd as fm

E, K, F = 8, 64, 32


def args(dtype, layout):
    n1, n2 = (E * 2 * F, K // 32), (E * K, F // 32)
    shape = (lambda n: fm.mx_k4_shape(*n)) if layout == fm.SCALE_E8M0_K4 else (lambda n: n)
    z = lambda *s: torch.zeros(*s, dtype=torch.uint8)
    return dict(x=torch.zeros(4, K, dtype=torch.bfloat16), ids=torch.zeros(4, 2, dtype=torch.int32), weights=torch.zeros(4, 2),
                w1=z(E, 2 * F, K), w1_scale=z(shape(n1)).view(dtype), w2=z(E, K, F), w2_scale=z(shape(n2)).view(dtype),
                scale_kind=layout)


@pytest.mark.parametrize("layout", [fm.SCALE_E8M0, fm.SCALE_E8M0_K4])
@pytest.mark.parametrize("dtype", [torch.uint8, torch.float8_e8m0fnu])
def test_taken(dtype, layout):
    with pytest.raises(ValueError, match="GPU tensors"):     # the last check before a launch
        fm.moe_few_tokens(**args(dtype, layout))


@pytest.mark.parametrize("name", ["w1_scale", "w2_scale"])
def test_refused(name):
    a = args(torch.uint8, fm.SCALE_E8M0)
    for bad in (a[name].view(torch.float8_e4m3fn), a[name].float(), a[name][:-1]):
        with pytest.raises(ValueError, match=name):
            fm.moe_few_tokens(**dict(a, **{name: bad}))
    with pytest.raises(ValueError, match="w1_scale"):        # e8m0 scales where fp32 ones are named
        fm.moe_few_tokens(**dict(args(torch.float8_e8m0fnu, fm.SCALE_E8M0), scale_kind=fm.SCALE_F32))


@pytest.mark.gpu
@pytest.mark.parametrize("layout", [fm.SCALE_E8M0, fm.SCALE_E8M0_K4])
def test_same_bytes_same_answer(layout):
    g = torch.Generator("cuda").manual_seed(3)
    a = {k: v.cuda() if torch.is_tensor(v) else v for k, v in args(torch.uint8, layout).items()}
    a["x"].normal_(generator=g)
    a["weights"].normal_(generator=g)
    for k in ("w1", "w2"):
        a[k].random_(0, 0x7F, generator=g)
    for k in ("w1_scale", "w2_scale"):
        a[k].random_(110, 118, generator=g)
    y = fm.moe_few_tokens(**a)
    assert torch.isfinite(y).all() and (y != 0).any()
    e8 = torch.float8_e8m0fnu
    assert torch.equal(y, fm.moe_few_tokens(**dict(a, w1_scale=a["w1_scale"].view(e8), w2_scale=a["w2_scale"].view(e8))))
