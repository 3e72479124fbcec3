"""The norm's rowwise scale and codes are the documented fp32 operations bit for bit: f = (s * gamma) * rstd,
scale = fmax / max(amax |f|, 1e-12), code = enc(clamp(f * scale)), each operation rounded once.

With bf16 rows and a bf16 gamma the products s * gamma are exact, and many scaled values lie on the border between two codes:
there the operations' roundings decide, and a form that takes them in another order answers otherwise."""
import numpy as np
import pytest

import mxfp8_quantized_moe_amd as fm
from oracle import codec as oc
from oracle.quant import bf16_to_f32
from oracle.swiglu import round_bf16
from gpu_helpers import note, bf16_dev, host, assert_bytes_equal, assert_f32_bits_equal

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("codec", [0, 1])
@pytest.mark.parametrize("R,C", [(700, 2056), (600, 4096), (16, 4096), (900, 512)])
def test_codes_are_the_documented_operations(R, C, codec):
    note(f"rmsnorm_quantize_rowwise operations {R}x{C} codec {codec}")
    rng = np.random.default_rng(R + C + codec)
    x = round_bf16(rng.standard_normal((R, C)))
    gamma = round_bf16(1 + 0.2 * rng.standard_normal(C))
    xd, gd = bf16_dev(x), bf16_dev(gamma)
    h, q, scale, rstd, _ = fm.rmsnorm_quantize_rowwise(xd, gd, 1e-6, codec=codec)
    f = (bf16_to_f32(x) * bf16_to_f32(gamma)) * host(rstd)[:, None]
    assert f.dtype == np.float32
    amax = np.maximum(np.abs(f).max(axis=1), np.float32(1e-12))
    sc = np.float32(oc.FMAX[codec]) / amax
    assert_f32_bits_equal(host(scale), sc, "scale")
    fmax = np.float32(oc.FMAX[codec])
    y = np.clip(f * sc[:, None], -fmax, fmax)
    assert_bytes_equal(host(q), oc.encode_nearest(y, codec), "codes")
    assert_bytes_equal(host(h), round_bf16(f.astype(np.float64)), "h")
    for _ in range(3):
        again = fm.rmsnorm_quantize_rowwise(xd, gd, 1e-6, codec=codec)
        assert all((a.view(b.dtype) == b).all() for a, b in zip(again[:4], (h, q, scale, rstd)))
