"""The MX recipe's backward from the kept input in a graph: both dual forms beside the product that reads one, replayed on new
inputs between eager calls and on a second stream; codes and scales kept as torch's 8-bit types."""
import numpy as np
import pytest
import torch

import mxfp8_quantized_moe_amd as fm
from oracle import quant as oq
from oracle.swiglu import round_bf16
from gpu_helpers import note, bf16_dev, i32_dev, u8_dev

pytestmark = pytest.mark.gpu


def test_step():
    note("kept SwiGLU, MX forms captured")
    rng = np.random.default_rng(12)
    R, F, K, E = 210, 128, 256, 3
    offs = i32_dev([64, 130, R])
    wq, ws, _ = fm.quantize_mx(bf16_dev(round_bf16(0.1 * rng.standard_normal((E * K, 2 * F)))), layout=fm.MX_LAYOUT_K4)

    def step(da2, hq, hs):
        _, q, s, q_t, s_t, pad = fm.swiglu_quantize_mx_dual_saved(hq, hs, offs)
        _, dq, ds, dq_t, ds_t, dpad = fm.swiglu_backward_quantize_mx_dual_saved(da2, hq, hs, offs)
        dx = fm.grouped_mm_scaled(fm.GROUPED_M, dq, fm.OPD_E4M3FN, ds, wq, fm.OPD_E4M3FN, ws, fm.SCALE_E8M0_K4, offs, E, R, K, 2 * F)
        return q, s, q_t, s_t, pad, dq, ds, dq_t, ds_t, dpad, dx

    inputs = []
    for _ in range(3):
        hq, hs = oq.quantize_mx_lastdim(round_bf16(2 * rng.standard_normal((R, 2 * F))), 0)
        inputs.append((bf16_dev(round_bf16(1e-3 * rng.standard_normal((R, F)))), u8_dev(hq), u8_dev(hs)))
    same = lambda a, b: all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))
    want = [[t.clone() for t in step(*v)] for v in inputs]
    typed = (inputs[0][0], inputs[0][1].view(torch.float8_e4m3fn), inputs[0][2].view(torch.float8_e8m0fnu))
    assert same(step(*typed), want[0])
    held = [t.clone() for t in inputs[0]]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step(*held)
    for i in (0, 1, 2, 1):
        for a, b in zip(held, inputs[i]):
            a.copy_(b)
        torch.cuda.synchronize()
        g.replay()
        other = fm.swiglu_backward_quantize_mx_dual_saved(*inputs[2], offs, stream=side)
        torch.cuda.synchronize()
        assert same(out, want[i])
        assert same(other[1:6], want[2][5:10])
        step(*inputs[0])
