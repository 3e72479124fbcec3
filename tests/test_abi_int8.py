"""The integer codec and operands at the C ABI: where they are taken and where refused (no GPU)."""
import pytest

from mxfp8_quantized_moe_amd import _lib as L

P = 0x10000


@pytest.fixture(scope="module")
def lib():
    return L.lib()


def mm(lib, mode=0, af=L.OPD_INT8, bf=L.OPD_INT8, sk=0, M=64, N=64, K=64, a=P, sa=P, out=P, offs=P, E=2):
    return lib.grouped_mm_scaled(mode, a, af, sa, P, bf, P, sk, offs, E, M, N, K, out, 0, None)


def test_product_refusals(lib):
    assert mm(lib, mode=1) == L.ERR_UNSUPPORTED                       # the weight gradient has no integer form
    assert mm(lib, af=L.OPD_E4M3FN) == L.ERR_UNSUPPORTED              # mixed operands
    assert mm(lib, bf=L.OPD_BF16) == L.ERR_UNSUPPORTED
    for sk in (L.SCALE_E8M0, L.SCALE_NONE, L.SCALE_E8M0_K4):
        assert mm(lib, sk=sk) == L.ERR_UNSUPPORTED
    assert mm(lib, K=131072) == L.ERR_UNSUPPORTED                     # the sum could leave 32 bits
    assert mm(lib, K=72) == L.ERR_ALIGN
    assert mm(lib, af=5, bf=5) == L.ERR_ENUM
    assert mm(lib, a=None) == L.ERR_NULL
    assert mm(lib, sa=None) == L.ERR_NULL
    assert mm(lib, sa=P + 1) == L.ERR_ALIGN
    assert mm(lib, out=P + 8) == L.ERR_ALIGN
    assert mm(lib, offs=None) == L.ERR_NULL
    assert mm(lib, M=-1) == L.ERR_SHAPE


def test_codec_where_it_is_taken(lib):
    i8 = L.INT8   # accepted: the next check answers
    assert lib.quantize_rowwise(None, 4, 16, 16, i8, P, P, None) == L.ERR_NULL
    assert lib.swiglu_quantize_rowwise(None, 4, 16, 32, i8, P, P, P, None) == L.ERR_NULL
    assert lib.moe_permute_quantized(None, P, 4, 32, 2, P, 8, i8, P, P, None) == L.ERR_NULL
    assert lib.moe_permute_rowwise(None, 4, 16, 2, P, 8, i8, P, P, P, None) == L.ERR_NULL
    assert lib.rmsnorm_quantize_rowwise(P, None, None, 1, 4, 64, 64, 64, 1e-6, i8, None, P, P, P + 1, P, None) == L.ERR_ALIGN


def test_codec_where_it_is_refused(lib):
    i8 = L.INT8
    assert lib.swiglu_backward_quantize_rowwise(P, P, 4, 16, 32, i8, P, P, P, None) == L.ERR_ENUM
    assert lib.quantize_colwise(P, 1, 64, 16, P, 4, i8, P, 64, P, None) == L.ERR_ENUM
    assert lib.quantize_tensorwise(P, 1, 4, 16, i8, P, P, 16, P, 4, P, None) == L.ERR_ENUM
    assert lib.quantize_blockwise(P, 1, 4, 16, 1, i8, P, P, None) == L.ERR_ENUM
    assert lib.quantize_blockwise_tokens(P, 64, 16, P, 2, i8, P, 64, P, None) == L.ERR_ENUM
    assert lib.moe_combine_backward(P, P, 8, P, P, P, 4, 2, 16, i8, P, P, P, P, None) == L.ERR_ENUM
    assert lib.fp8moe_encode_f32(P, 16, i8, P, None) == L.ERR_ENUM
