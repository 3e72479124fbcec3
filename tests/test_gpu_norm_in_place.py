"""The sum written over x or over the residual, in every form of the norm kernel: the results of separate arrays, bit for bit."""
import numpy as np
import pytest
import torch

import mxfp8_quantized_moe_amd as fm
from oracle.swiglu import round_bf16
from gpu_helpers import note, bf16_dev

pytestmark = pytest.mark.gpu

# columns for each count of threads and chunks a row takes, few rows and many
SHAPES = [(40, 128), (40, 256), (40, 512), (40, 1024), (40, 2048), (600, 2560), (600, 4096), (600, 6144), (600, 8192), (600, 16384),
          (40, 2560), (40, 8192), (40, 16384), (1, 64), (1, 16384)]


@pytest.mark.parametrize("R,C", SHAPES)
def test_every_form(R, C):
    note(f"rmsnorm in place {R}x{C}")
    rng = np.random.default_rng(R + C)
    x, res = bf16_dev(round_bf16(rng.standard_normal((R, C)))), bf16_dev(round_bf16(rng.standard_normal((R, C))))
    gamma = torch.from_numpy((1 + 0.2 * rng.standard_normal(C)).astype(np.float32)).to(x.device)
    forms = [lambda a, b, s: fm.rmsnorm_quantize_rowwise(a, gamma, residual=b, sum_out=s),
             lambda a, b, s: fm.rmsnorm_quantize_rowwise(a, gamma, residual=b, sum_out=s, codec=fm.E4M3FNUZ),
             lambda a, b, s: fm.rmsnorm_quantize_rowwise(a, gamma, residual=b, sum_out=s, codes=False),
             lambda a, b, s: fm.rmsnorm_quantize_mx(a, gamma, residual=b, sum_out=s),
             lambda a, b, s: fm.rmsnorm_quantize_mx(a, None, residual=b, sum_out=s, rule=fm.MX_CEIL, layout=fm.MX_LAYOUT_K4)]
    for form in forms:
        want = form(x, res, None)
        for over in (0, 1):
            a = [x.clone(), res.clone()]
            got = form(a[0], a[1], a[over])
            assert got[4] is a[over]
            assert all(u is None if v is None else torch.equal(u, v) for u, v in zip(got, want))
            assert torch.equal(a[1 - over], (x, res)[1 - over])      # the other one stays
        both = form(x, x, None)
        c = x.clone()
        got = form(c, c, c)                                          # x + x over x
        assert all(u is None if v is None else torch.equal(u, v) for u, v in zip(got, both))
