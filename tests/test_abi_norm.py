"""Refusals of the norm's entry points, on the host: no HIP call is reached and no fake pointer is read."""
import math

import pytest
import torch

import mxfp8_quantized_moe_amd as fm
from mxfp8_quantized_moe_amd import _lib as L

P, MIS = 0x10000, 0x10001


@pytest.fixture(scope="module")
def lib():
    return L.lib()


def refused(f, ok, **kw):
    a = dict(ok, **kw)
    return f(*a.values())


def forward_args(**kw):
    return dict(x=P, res=P, gamma=P, gt=1, rows=4, cols=64, ld=64, ld_r=64, eps=1e-6, **kw)


def test_forward_rejections(lib):
    rw = forward_args(codec=0, sum=P, h=P, q=P, scale=P, rstd=P, stream=None)
    mx = forward_args(rule=0, layout=0, sum=P, h=P, q=P, scale=P, rstd=P, stream=None)
    for f, ok in ((lib.rmsnorm_quantize_rowwise, rw), (lib.rmsnorm_quantize_mx, mx)):
        assert refused(f, ok, gt=2) == L.ERR_ENUM
        assert refused(f, ok, rows=-1) == L.ERR_SHAPE
        assert refused(f, ok, cols=0) == L.ERR_SHAPE
        assert refused(f, ok, ld=32) == L.ERR_SHAPE
        assert refused(f, ok, ld_r=32) == L.ERR_SHAPE
        assert refused(f, ok, rows=1 << 40) == L.ERR_SHAPE
        assert refused(f, ok, cols=16392, ld=16392, ld_r=16392) == L.ERR_UNSUPPORTED
        for eps in (0.0, -1.0, math.inf, math.nan):
            assert refused(f, ok, eps=eps) == L.ERR_VALUE
        for p in ("x", "sum"):
            assert refused(f, ok, **{p: None}) == L.ERR_NULL
        assert refused(f, ok, q=None) == L.ERR_NULL            # codes and scales come together
        assert refused(f, ok, scale=None) == L.ERR_NULL
        assert refused(f, ok, cols=60) == L.ERR_ALIGN
        assert refused(f, ok, ld=68) == L.ERR_ALIGN
        assert refused(f, ok, ld_r=68) == L.ERR_ALIGN
        for p in ("x", "res", "gamma", "sum", "h", "q", "rstd"):
            assert refused(f, ok, **{p: MIS}) == L.ERR_ALIGN, p
        # in place only where rows lie as the sum's do: else a row's sum would land in rows not read yet
        assert refused(f, ok, ld=72) == L.ERR_SHAPE
        assert refused(f, ok, ld=72, x=2 * P, sum=2 * P, res=3 * P) == L.ERR_SHAPE
        assert refused(f, ok, x=2 * P, ld_r=72) == L.ERR_SHAPE
        assert refused(f, ok, rows=0, x=None, res=None, sum=None, h=None, q=None, scale=None, rstd=None) == L.OK
    assert refused(lib.rmsnorm_quantize_rowwise, rw, codec=2) == L.ERR_ENUM
    assert refused(lib.rmsnorm_quantize_rowwise, rw, scale=P + 2) == L.ERR_ALIGN
    assert refused(lib.rmsnorm_quantize_mx, mx, rule=2) == L.ERR_ENUM
    assert refused(lib.rmsnorm_quantize_mx, mx, layout=2) == L.ERR_ENUM
    assert refused(lib.rmsnorm_quantize_mx, mx, cols=40) == L.ERR_ALIGN     # cols % 32
    assert refused(lib.rmsnorm_quantize_mx, mx, q=None, scale=None) == L.ERR_NULL


def test_backward_rejections(lib):
    ok = dict(dh=P, s=P, rstd=P, gamma=P, gt=0, dsum=P, rows=4, cols=64, dx=P, dgamma=P, ws=P, stream=None)
    f = lib.rmsnorm_backward
    assert refused(f, ok, gt=7) == L.ERR_ENUM
    assert refused(f, ok, rows=-1) == L.ERR_SHAPE
    assert refused(f, ok, cols=0) == L.ERR_SHAPE
    assert refused(f, ok, cols=16392) == L.ERR_UNSUPPORTED
    for p in ("dh", "s", "rstd", "dx", "ws"):
        assert refused(f, ok, **{p: None}) == L.ERR_NULL, p
    assert refused(f, ok, cols=60) == L.ERR_ALIGN
    for p in ("dh", "s", "rstd", "gamma", "dsum", "dx", "dgamma", "ws"):
        assert refused(f, ok, **{p: MIS}) == L.ERR_ALIGN, p
    assert refused(f, ok, rows=0, dh=None, s=None, rstd=None, dx=None, dgamma=None, ws=None) == L.OK
    assert lib.rmsnorm_backward_workspace_bytes(-1, 64) == -1
    assert lib.rmsnorm_backward_workspace_bytes(4, 16392) == -1
    assert lib.rmsnorm_backward_workspace_bytes(0, 64) == 0
    assert lib.rmsnorm_backward_workspace_bytes(1, 64) >= 4 * 64
    assert lib.fp8moe_status_string(L.ERR_VALUE) not in (b"ok", b"unknown status")


def test_binding_refusals():
    """Wrong types, shapes, strides and places raise before anything is allocated or launched."""
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    for fn in (fm.rmsnorm_quantize_rowwise, fm.rmsnorm_quantize_mx):
        for bad in (x.float(), x[0], x.t(), x[:, ::2], x.unsqueeze(0), x[:1].expand(4, 64)):
            with pytest.raises(ValueError, match="x "):
                fn(bad)
        with pytest.raises(ValueError, match="residual"):
            fn(x, residual=x[:3])
        with pytest.raises(ValueError, match="residual"):
            fn(x, residual=x.half())
        for gamma in (torch.ones(63), torch.ones(64, dtype=torch.float64), torch.ones(1, 64), torch.ones(128)[::2]):
            with pytest.raises(ValueError, match="gamma"):
                fn(x, gamma)
        with pytest.raises(ValueError, match="GPU"):
            fn(x)
    r = torch.ones(4)
    for kw in (dict(dh=x[:3]), dict(s=x.float()), dict(rstd=r[:3]), dict(rstd=r.double()), dict(dsum=x[:, :32]),
               dict(dh=torch.zeros(4, 72, dtype=torch.bfloat16)[:, :64]), dict(gamma=torch.ones(32)), dict()):
        a = dict(dict(dh=x, s=x, rstd=r), **kw)
        with pytest.raises(ValueError):
            fm.rmsnorm_backward(**a)
