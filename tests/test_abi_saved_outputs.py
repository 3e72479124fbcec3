"""The MX forms from the kept SwiGLU input refuse outputs of another size, type, stride or device (no GPU)."""
import pytest
import torch

import mxfp8_quantized_moe_amd as fm

R, F, E, RP = 64, 128, 3, 192
U8 = torch.uint8


def outputs(C, layout, bf16):
    sc = fm.mx_k4_shape if layout == fm.MX_LAYOUT_K4 else lambda rows, nb: (rows, nb)
    return {bf16: torch.zeros(R, C, dtype=torch.bfloat16), "q": torch.zeros(R, C, dtype=U8),
            "scale": torch.zeros(sc(R, C // 32), dtype=U8), "q_t": torch.zeros(C, RP, dtype=U8),
            "scale_t": torch.zeros(sc(C, RP // 32), dtype=U8), "offs_pad": torch.zeros(E, dtype=torch.int32)}


@pytest.mark.parametrize("layout", [fm.MX_LAYOUT_ROWS, fm.MX_LAYOUT_K4])
@pytest.mark.parametrize("bwd", [False, True])
def test_outputs(bwd, layout):
    hq, hs = torch.zeros(R, 2 * F, dtype=U8), torch.zeros(R, 2 * F // 32, dtype=U8)
    args = (hq, hs, torch.zeros(E, dtype=torch.int32))
    f, C, bf16 = fm.swiglu_quantize_mx_dual_saved, F, "a2"
    if bwd:
        f, C, bf16 = fm.swiglu_backward_quantize_mx_dual_saved, 2 * F, "dh1"
        args = (torch.zeros(R, F, dtype=torch.bfloat16),) + args
    good = outputs(C, layout, bf16)
    for name, t in good.items():
        wrong_type = {torch.bfloat16: torch.float16, U8: torch.int16, torch.int32: torch.int64}[t.dtype]
        bad = [t[:-1], t.to(wrong_type), torch.zeros(*t.shape, 2, dtype=t.dtype)[..., 0], t.to("meta")]
        if t.dim() > 1:
            bad.append(t[:, :-1].contiguous())
        for b in bad:
            with pytest.raises(ValueError, match=rf"mx_dual_saved: {name} must be"):
                f(*args, rows_pad=RP, layout=layout, **dict(good, **{name: b}))
    with pytest.raises(ValueError, match="mx_dual_saved: q_t must be"):   # another padding than the outputs have
        f(*args, rows_pad=RP + 32, layout=layout, **good)
    as_float = dict(good, q=good["q"].view(torch.float8_e4m3fn), scale=good["scale"].view(torch.float8_e8m0fnu))
    for kw in (good, as_float, {}):
        with pytest.raises(ValueError, match="GPU tensors"):
            f(*args, rows_pad=RP, layout=layout, **kw)
