"""The kept SwiGLU from 2048 rows on, where rows of 17 to 192 chunks of eight columns go to 16 threads with two chunks each or to
a wave with two or three: short last chunks, rows that end inside a workgroup."""
import pytest

import test_gpu_saved as base

pytestmark = pytest.mark.gpu

SIZES = [(2051, 160), (2063, 256), (2048, 192), (2050, 544), (2051, 1024), (2049, 800), (2049, 1056), (2050, 1408), (2051, 1536)]


@pytest.mark.parametrize("codec,rule,pad", [(0, 0, 0), (1, 1, 40)])
@pytest.mark.parametrize("R,F", SIZES)
def test_save(R, F, codec, rule, pad):
    base.test_save(R, F, codec, rule, pad)


@pytest.mark.parametrize("codec", [0, 1])
@pytest.mark.parametrize("R,F", SIZES)
def test_saved_backward(R, F, codec):
    base.test_saved_backward(R, F, codec)
