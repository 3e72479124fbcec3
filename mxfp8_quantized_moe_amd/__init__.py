"""MI355X-native FP8 MoE quantization + grouped GEMM (thin Python binding).

Every function here marshals torch tensors to device pointers and calls the
C ABI of libfp8moe.so (include/fp8moe.h) on the current HIP stream; every step
of the computation runs in the library's HIP kernels.  Outputs not supplied
by the caller are allocated with torch (device memory plumbing only).  There is
no CPU or eager fallback: a missing library or a rejected argument raises.
"""
from __future__ import annotations

import contextlib

import torch

from . import _lib
from ._lib import (E4M3FN, E4M3FNUZ, INT8, MX_FLOOR_OCP, MX_CEIL, MX_LAYOUT_ROWS, MX_LAYOUT_K4, GROUPED_M, GROUPED_K,
                   OPD_E4M3FN, OPD_E4M3FNUZ, OPD_BF16, OPD_INT8, SCALE_F32, SCALE_E8M0, SCALE_NONE, SCALE_E8M0_K4,
                   OUT_BF16, OUT_F32, GATE_SOFTMAX, GATE_SIGMOID,
                   Fp8MoeError)

__all__ = ["quantize_rowwise", "quantize_colwise", "quantize_mx", "quantize_mx_rows_bound",
           "grouped_mm_scaled", "encode_f32", "default_codec", "E4M3FN", "E4M3FNUZ", "INT8", "MX_FLOOR_OCP",
           "MX_CEIL", "MX_LAYOUT_ROWS", "MX_LAYOUT_K4", "GROUPED_M", "GROUPED_K", "OPD_E4M3FN", "OPD_E4M3FNUZ",
           "OPD_BF16", "OPD_INT8", "SCALE_F32", "SCALE_E8M0", "SCALE_NONE", "SCALE_E8M0_K4", "OUT_BF16", "OUT_F32",
           "mx_k4_shape", "quantize_mx_dual", "swiglu_quantize_mx_dual", "swiglu_backward_quantize_mx_dual",
           "moe_permute_quantize_mx_dual", "moe_permute_quantize_colwise",
           "Fp8MoeError", "swiglu_quantize_rowwise",
           "swiglu_backward_quantize_rowwise", "moe_route", "moe_route_noalloc", "moe_route_rows_bound", "moe_route_workspace_bytes", "moe_permute", "moe_combine",
           "moe_permute_rowwise", "moe_combine_backward",
           "quantize_tensorwise", "moe_permute_quantized", "quantize_blockwise", "grouped_mm_blockwise",
           "quantize_blockwise_tokens", "grouped_mm_blockwise_k",
           "rmsnorm_quantize_rowwise", "rmsnorm_quantize_mx", "rmsnorm_backward", "rmsnorm_backward_workspace_bytes",
           "GATE_SOFTMAX", "GATE_SIGMOID", "moe_gate", "moe_gate_balance", "moe_gate_backward", "moe_balance_loss",
           "moe_balance_loss_backward", "moe_balance_workspace_bytes", "moe_few_tokens", "moe_few_tokens_workspace_bytes",
           "swiglu_quantize_rowwise_save", "swiglu_backward_quantize_rowwise_saved", "swiglu_quantize_mx_dual_saved",
           "swiglu_backward_quantize_mx_dual_saved"]


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    if stream is None:   # the raw handle: torch.cuda.current_stream builds a Stream object first (2.7 us instead of 0.3)
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return stream.cuda_stream


def _bits(x: torch.Tensor) -> torch.Tensor:
    """bf16 tensors pass as their 16-bit patterns; int16/uint16 pass through."""
    if x.dtype == torch.bfloat16:
        return x
    if x.dtype in (torch.int16, torch.uint16):
        return x
    raise TypeError(f"expected bf16 (or its 16-bit pattern), got {x.dtype}")


def _codes(codec):
    """The dtype of a codec's codes."""
    return torch.int8 if codec == INT8 else torch.uint8


def quantize_rowwise(x, codec=E4M3FN, q=None, scale=None, stream=None):
    """x [R, C] bf16 (row stride may exceed C) -> (q uint8 [R, C], scale f32 [R]); codec=INT8 gives int8 codes."""
    x = _bits(x)
    R, C = x.shape
    if x.numel() and x.stride(1) != 1:
        raise ValueError("quantize_rowwise needs unit stride along the last dim")
    ld_x = x.stride(0) if x.numel() else C
    q = torch.empty((R, C), dtype=_codes(codec), device=x.device) if q is None else q
    scale = torch.empty((R,), dtype=torch.float32, device=x.device) if scale is None else scale
    _lib.check("quantize_rowwise", _lib.lib().quantize_rowwise(
        _ptr(x), R, C, ld_x, codec, _ptr(q), _ptr(scale), _stream(stream)))
    return q, scale


def quantize_colwise(x, offs=None, codec=E4M3FN, q_t=None, scale=None, ld_q=None, stream=None):
    """Grouped 2D: x [M, C] + offs [E] -> (q_t uint8 phys [C, ld_q], scale [E, C]).
    Batched 3D: x [B, R, C] -> (q_t uint8 phys [B, C, ld_q], scale [B, C]).
    ld_q defaults to the row count rounded up to a multiple of 16 (the ABI's alignment)."""
    x = _bits(x).contiguous()
    if offs is not None:
        M, C = x.shape
        B, R, E = 1, M, offs.numel()
        ld_q = ld_q or (M + 15) // 16 * 16
        q_t = torch.empty((C, ld_q), dtype=torch.uint8, device=x.device) if q_t is None else q_t
        scale = torch.empty((E, C), dtype=torch.float32, device=x.device) if scale is None else scale
    else:
        B, R, C = x.shape
        E = 0
        ld_q = ld_q or (R + 15) // 16 * 16
        q_t = torch.empty((B, C, ld_q), dtype=torch.uint8, device=x.device) if q_t is None else q_t
        scale = torch.empty((B, C), dtype=torch.float32, device=x.device) if scale is None else scale
    _lib.check("quantize_colwise", _lib.lib().quantize_colwise(
        _ptr(x), B, R, C, _ptr(offs), E, codec, _ptr(q_t), ld_q, _ptr(scale), _stream(stream)))
    return q_t, scale


def moe_permute_quantize_colwise(x, src, topk, offs, weights=None, codec=E4M3FN, q_t=None, scale=None, ld_q=None,
                                 stream=None):
    """x bf16 [T, C] (token rows, or the output gradient dy), src int32 [R], offs int32 [E] from moe_route,
    weights f32 [T, topk] or None -> (q_t uint8 phys [C, ld_q], scale [E, C]): quantize_colwise of the gathered
    rows x[src[r] // topk] (times weights[src[r]] when given, rounded to bf16), which never go to memory."""
    x = _bits(x).contiguous()
    T, C = x.shape
    R, E = src.numel(), offs.numel()
    if weights is not None:
        weights = weights.contiguous()
        if weights.dtype != torch.float32 or weights.numel() != T * topk:
            raise ValueError("moe_permute_quantize_colwise: weights f32 [T, topk]")
    ld_q = ld_q or (R + 15) // 16 * 16
    q_t = torch.empty((C, ld_q), dtype=torch.uint8, device=x.device) if q_t is None else q_t
    scale = torch.empty((E, C), dtype=torch.float32, device=x.device) if scale is None else scale
    _lib.check("moe_permute_quantize_colwise", _lib.lib().moe_permute_quantize_colwise(
        _ptr(x), T, C, topk, _ptr(src), _ptr(weights), R, _ptr(offs), E, codec, _ptr(q_t), ld_q, _ptr(scale),
        _stream(stream)))
    return q_t, scale


def quantize_mx_rows_bound(rows: int, n_groups: int) -> int:
    return int(_lib.lib().quantize_mx_rows_bound(rows, n_groups))


def mx_k4_shape(rows: int, n_blocks: int):
    """Shape of an e8m0 scale matrix of `rows` rows and `n_blocks` 32-blocks per row in the K4
    layout: [ceil(n_blocks / 4), rows, 4]."""
    return ((n_blocks + 3) // 4, rows, 4)


def quantize_mx(x, axis=1, offs=None, rule=MX_FLOOR_OCP, rows_pad=None, q=None, scale=None,
                offs_pad=None, layout=MX_LAYOUT_ROWS, stream=None):
    """MXFP8.  axis=1: x [R, C] -> (q [R, C], e8m0 [R, C/32], None).
    axis=0 without offs: x [B, R, C] -> (q phys [B, C, R], e8m0 [B, C, R/32], None).
    axis=0 with offs: x [M, C] -> (q phys [C, rows_pad], e8m0 [C, rows_pad/32], offs_pad [E]).
    layout=MX_LAYOUT_K4: e8m0 in the K4 layout instead, shape mx_k4_shape(scale rows, blocks) with
    scale rows R (axis 1), B*C (axis 0 without offs), C (axis 0 with offs)."""
    x = _bits(x).contiguous()
    dev = x.device
    k4 = layout == MX_LAYOUT_K4

    def sc_empty(rows_major_shape, n_rows, n_blocks):
        shape = mx_k4_shape(n_rows, n_blocks) if k4 else rows_major_shape
        return torch.empty(shape, dtype=torch.uint8, device=dev)

    if axis == 1:
        C = x.shape[-1]
        R = x.numel() // max(C, 1)
        q = torch.empty(tuple(x.shape), dtype=torch.uint8, device=dev) if q is None else q
        scale = sc_empty(tuple(x.shape[:-1]) + (C // 32,), R, C // 32) if scale is None else scale
        st = _lib.lib().quantize_mx(_ptr(x), 1, R, C, 1, None, 0, rule, layout, _ptr(q), _ptr(scale), 0, None,
                                    _stream(stream))
        _lib.check("quantize_mx", st)
        return q, scale, None
    if offs is None:
        B, R, C = x.shape
        q = torch.empty((B, C, R), dtype=torch.uint8, device=dev) if q is None else q
        scale = sc_empty((B, C, R // 32), B * C, R // 32) if scale is None else scale
        st = _lib.lib().quantize_mx(_ptr(x), B, R, C, 0, None, 0, rule, layout, _ptr(q), _ptr(scale), R, None,
                                    _stream(stream))
        _lib.check("quantize_mx", st)
        return q, scale, None
    M, C = x.shape
    E = offs.numel()
    rows_pad = rows_pad or quantize_mx_rows_bound(M, E)
    q = torch.empty((C, rows_pad), dtype=torch.uint8, device=dev) if q is None else q
    scale = sc_empty((C, rows_pad // 32), C, rows_pad // 32) if scale is None else scale
    offs_pad = torch.empty((E,), dtype=torch.int32, device=dev) if offs_pad is None else offs_pad
    st = _lib.lib().quantize_mx(_ptr(x), 1, M, C, 0, _ptr(offs), E, rule, layout, _ptr(q), _ptr(scale), rows_pad,
                                _ptr(offs_pad), _stream(stream))
    _lib.check("quantize_mx", st)
    return q, scale, offs_pad


def quantize_mx_dual(x, offs=None, rule=MX_FLOOR_OCP, rows_pad=None, q=None, scale=None, q_t=None, scale_t=None,
                     offs_pad=None, layout=MX_LAYOUT_ROWS, stream=None):
    """Both MXFP8 forms from one read: (q, scale) as quantize_mx(x viewed [B*R, C], axis=1) and
    (q_t, scale_t, offs_pad) as quantize_mx(x, axis=0, offs).  x is [B, R, C] without offs, [M, C] with."""
    x = _bits(x).contiguous()
    dev = x.device
    k4 = layout == MX_LAYOUT_K4

    def sc_empty(rows_major_shape, n_rows, n_blocks):
        shape = mx_k4_shape(n_rows, n_blocks) if k4 else rows_major_shape
        return torch.empty(shape, dtype=torch.uint8, device=dev)

    if offs is None:
        B, R, C = x.shape
        E, rp, offs_pad = 0, R, None
        q_t = torch.empty((B, C, R), dtype=torch.uint8, device=dev) if q_t is None else q_t
        scale_t = sc_empty((B, C, R // 32), B * C, R // 32) if scale_t is None else scale_t
    else:
        (M, C), B = x.shape, 1
        R = M
        E = offs.numel()
        rp = rows_pad or quantize_mx_rows_bound(M, E)
        q_t = torch.empty((C, rp), dtype=torch.uint8, device=dev) if q_t is None else q_t
        scale_t = sc_empty((C, rp // 32), C, rp // 32) if scale_t is None else scale_t
        offs_pad = torch.empty((E,), dtype=torch.int32, device=dev) if offs_pad is None else offs_pad
    q = torch.empty((B * R, C), dtype=torch.uint8, device=dev) if q is None else q
    scale = sc_empty((B * R, C // 32), B * R, C // 32) if scale is None else scale
    st = _lib.lib().quantize_mx_dual(_ptr(x), B, R, C, _ptr(offs), E, rule, layout, _ptr(q), _ptr(scale), _ptr(q_t),
                                     _ptr(scale_t), rp, _ptr(offs_pad), _stream(stream))
    _lib.check("quantize_mx_dual", st)
    return q, scale, q_t, scale_t, offs_pad


def _mx_dual_outputs(R, C, offs, rows_pad, q, scale, q_t, scale_t, offs_pad, layout, dev):
    k4 = layout == MX_LAYOUT_K4
    E = offs.numel()
    rp = rows_pad or quantize_mx_rows_bound(R, E)
    sc_shape = lambda rows_major, n_rows, n_blocks: mx_k4_shape(n_rows, n_blocks) if k4 else rows_major
    q = torch.empty((R, C), dtype=torch.uint8, device=dev) if q is None else q
    scale = torch.empty(sc_shape((R, C // 32), R, C // 32), dtype=torch.uint8, device=dev) if scale is None else scale
    q_t = torch.empty((C, rp), dtype=torch.uint8, device=dev) if q_t is None else q_t
    scale_t = torch.empty(sc_shape((C, rp // 32), C, rp // 32), dtype=torch.uint8, device=dev) \
        if scale_t is None else scale_t
    offs_pad = torch.empty((E,), dtype=torch.int32, device=dev) if offs_pad is None else offs_pad
    return rp, q, scale, q_t, scale_t, offs_pad


def moe_permute_quantize_mx_dual(x, src, topk, offs, weights=None, rule=MX_FLOOR_OCP, rows_pad=None, xg=None,
                                 q=None, scale=None, q_t=None, scale_t=None, offs_pad=None, layout=MX_LAYOUT_K4,
                                 stream=None):
    """x bf16 [T, C] (token rows, or the output gradient dy), src int32 [R], offs int32 [E] from moe_route,
    weights f32 [T, topk] or None -> (xg or None, q [R, C], scale, q_t [C, rows_pad], scale_t, offs_pad): both
    MX forms of the gathered rows x[src[r] // topk] (times weights[src[r]] when given, rounded to bf16);
    xg (bf16 [R, C]) is written only if passed."""
    x = _bits(x).contiguous()
    T, C = x.shape
    R = src.numel()
    if weights is not None:
        weights = weights.contiguous()
        if weights.dtype != torch.float32 or weights.numel() != T * topk:
            raise ValueError("moe_permute_quantize_mx_dual: weights f32 [T, topk]")
    rp, q, scale, q_t, scale_t, offs_pad = _mx_dual_outputs(R, C, offs, rows_pad, q, scale, q_t, scale_t, offs_pad,
                                                            layout, x.device)
    _lib.check("moe_permute_quantize_mx_dual", _lib.lib().moe_permute_quantize_mx_dual(
        _ptr(x), T, C, topk, _ptr(src), _ptr(weights), R, _ptr(offs), offs.numel(), rule, layout, _ptr(xg), _ptr(q),
        _ptr(scale), _ptr(q_t), _ptr(scale_t), rp, _ptr(offs_pad), _stream(stream)))
    return xg, q, scale, q_t, scale_t, offs_pad


def swiglu_quantize_mx_dual(h1, offs, rule=MX_FLOOR_OCP, rows_pad=None, a2=None, q=None, scale=None, q_t=None,
                            scale_t=None, offs_pad=None, layout=MX_LAYOUT_K4, stream=None):
    """h1 [R, 2F] bf16 (gate | up), offs int32 [E] -> (a2 or None, q [R, F], scale, q_t [F, rows_pad], scale_t,
    offs_pad): both MX forms of bf16(silu(gate) * up); a2 (bf16 [R, F]) is written only if passed."""
    h1 = _bits(h1)
    R, F2 = h1.shape
    if F2 % 2 or (h1.numel() and h1.stride(1) != 1):
        raise ValueError("swiglu_quantize_mx_dual needs an even column count and unit column stride")
    F = F2 // 2
    ld = h1.stride(0) if h1.numel() else F2
    rp, q, scale, q_t, scale_t, offs_pad = _mx_dual_outputs(R, F, offs, rows_pad, q, scale, q_t, scale_t, offs_pad,
                                                            layout, h1.device)
    _lib.check("swiglu_quantize_mx_dual", _lib.lib().swiglu_quantize_mx_dual(
        _ptr(h1), R, F, ld, _ptr(offs), offs.numel(), rule, layout, _ptr(a2), _ptr(q), _ptr(scale), _ptr(q_t),
        _ptr(scale_t), rp, _ptr(offs_pad), _stream(stream)))
    return a2, q, scale, q_t, scale_t, offs_pad


def swiglu_backward_quantize_mx_dual(da2, h1, offs, rule=MX_FLOOR_OCP, rows_pad=None, dh1=None, q=None, scale=None,
                                     q_t=None, scale_t=None, offs_pad=None, layout=MX_LAYOUT_K4, stream=None):
    """da2 [R, F], h1 [R, 2F] bf16, offs int32 [E] -> (dh1 or None, q [R, 2F], scale, q_t [2F, rows_pad], scale_t,
    offs_pad): both MX forms of SwiGLU's input gradient; dh1 (bf16 [R, 2F]) is written only if passed."""
    h1 = _bits(h1)
    da2 = _bits(da2).contiguous()
    R, F2 = h1.shape
    if F2 % 2 or (h1.numel() and h1.stride(1) != 1) or tuple(da2.shape) != (R, F2 // 2):
        raise ValueError("swiglu_backward_quantize_mx_dual: h1 [R, 2F] with unit column stride, da2 [R, F]")
    F = F2 // 2
    ld = h1.stride(0) if h1.numel() else F2
    rp, q, scale, q_t, scale_t, offs_pad = _mx_dual_outputs(R, F2, offs, rows_pad, q, scale, q_t, scale_t, offs_pad,
                                                            layout, h1.device)
    _lib.check("swiglu_backward_quantize_mx_dual", _lib.lib().swiglu_backward_quantize_mx_dual(
        _ptr(da2), _ptr(h1), R, F, ld, _ptr(offs), offs.numel(), rule, layout, _ptr(dh1), _ptr(q), _ptr(scale),
        _ptr(q_t), _ptr(scale_t), rp, _ptr(offs_pad), _stream(stream)))
    return dh1, q, scale, q_t, scale_t, offs_pad


def grouped_mm_scaled(mode, a, a_fmt, a_scale, b, b_fmt, b_scale, scale_kind, offs, n_groups, M, N, K,
                      out=None, out_dtype=OUT_BF16, stream=None):
    """See include/fp8moe.h.  GROUPED_M -> out [M, N]; GROUPED_K -> out [E, N, K]."""
    dev = a.device
    if out is None:
        shape = (M, N) if mode == GROUPED_M else (n_groups, N, K)
        out = torch.empty(shape, dtype=torch.bfloat16 if out_dtype == OUT_BF16 else torch.float32, device=dev)
    st = _lib.lib().grouped_mm_scaled(mode, _ptr(a), a_fmt, _ptr(a_scale), _ptr(b), b_fmt, _ptr(b_scale),
                                      scale_kind, _ptr(offs), n_groups, M, N, K, _ptr(out), out_dtype,
                                      _stream(stream))
    _lib.check("grouped_mm_scaled", st)
    return out


def swiglu_quantize_rowwise(h1, codec=E4M3FN, a2=None, q=None, scale=None, stream=None, codes=True):
    """h1 [R, 2F] bf16 (gate | up; row stride may exceed 2F) -> (a2 bf16 [R, F], q uint8 [R, F], scale f32 [R]);
    with codes=False only a2 is computed and q, scale are None."""
    h1 = _bits(h1)
    R, F2 = h1.shape
    if F2 % 2 or (h1.numel() and h1.stride(1) != 1):
        raise ValueError("swiglu_quantize_rowwise needs an even column count and unit column stride")
    F = F2 // 2
    ld = h1.stride(0) if h1.numel() else F2
    a2 = torch.empty((R, F), dtype=torch.bfloat16, device=h1.device) if a2 is None else a2
    if codes:
        q = torch.empty((R, F), dtype=_codes(codec), device=h1.device) if q is None else q
        scale = torch.empty((R,), dtype=torch.float32, device=h1.device) if scale is None else scale
    else:
        q = scale = None
    _lib.check("swiglu_quantize_rowwise", _lib.lib().swiglu_quantize_rowwise(
        _ptr(h1), R, F, ld, codec, _ptr(a2), _ptr(q), _ptr(scale), _stream(stream)))
    return a2, q, scale


def swiglu_backward_quantize_rowwise(da2, h1, codec=E4M3FN, dh1=None, q=None, scale=None, stream=None, codes=True):
    """da2 [R, F] bf16 and h1 [R, 2F] bf16 -> (dh1 bf16 [R, 2F], q uint8 [R, 2F], scale f32 [R]);
    with codes=False only dh1 is computed and q, scale are None."""
    h1 = _bits(h1)
    da2 = _bits(da2).contiguous()
    R, F2 = h1.shape
    if F2 % 2 or (h1.numel() and h1.stride(1) != 1) or tuple(da2.shape) != (R, F2 // 2):
        raise ValueError("swiglu_backward_quantize_rowwise: h1 [R, 2F] with unit column stride, da2 [R, F]")
    F = F2 // 2
    ld = h1.stride(0) if h1.numel() else F2
    dh1 = torch.empty((R, F2), dtype=torch.bfloat16, device=h1.device) if dh1 is None else dh1
    if codes:
        q = torch.empty((R, F2), dtype=torch.uint8, device=h1.device) if q is None else q
        scale = torch.empty((R,), dtype=torch.float32, device=h1.device) if scale is None else scale
    else:
        q = scale = None
    _lib.check("swiglu_backward_quantize_rowwise", _lib.lib().swiglu_backward_quantize_rowwise(
        _ptr(da2), _ptr(h1), R, F, ld, codec, _ptr(dh1), _ptr(q), _ptr(scale), _stream(stream)))
    return dh1, q, scale


def quantize_tensorwise(x, codec=E4M3FN, rowmajor=True, transposed=False, ld_q=None, n_scale=None, q=None,
                        q_t=None, scale=None, workspace=None, stream=None):
    """x bf16 [R, C] or [B, R, C] -> (q u8 [B*R, C] or None, q_t u8 [B, C, ld_q] or None, scale f32 [n_scale]).
    One scale for the whole tensor, repeated n_scale times (default: B*R, the row count); ld_q defaults to R
    rounded up to 16."""
    x = _bits(x).contiguous()
    B, R, C = (1, *x.shape) if x.dim() == 2 else tuple(x.shape)
    dev = x.device
    if rowmajor and q is None:
        q = torch.empty((B * R, C), dtype=torch.uint8, device=dev)
    if transposed:
        ld_q = (R + 15) // 16 * 16 if ld_q is None else ld_q   # rows of q_t start 16-byte aligned
        if q_t is None:
            q_t = torch.empty((B, C, ld_q), dtype=torch.uint8, device=dev)
    n_scale = max(B * R, 1) if n_scale is None else n_scale
    scale = torch.empty((n_scale,), dtype=torch.float32, device=dev) if scale is None else scale
    if workspace is None:
        workspace = torch.empty(int(_lib.lib().quantize_tensorwise_workspace_bytes()), dtype=torch.uint8, device=dev)
    _lib.check("quantize_tensorwise", _lib.lib().quantize_tensorwise(
        _ptr(x), B, R, C, codec, _ptr(q) if rowmajor else None, _ptr(q_t) if transposed else None,
        ld_q if transposed else 0, _ptr(scale), n_scale, _ptr(workspace), _stream(stream)))
    return (q if rowmajor else None), (q_t if transposed else None), scale


def quantize_blockwise(x, block_rows, codec=E4M3FN, q=None, scale=None, stream=None):
    """x bf16 [R, C] or [B, R, C] -> (q u8 of x's shape, scale f32 [B, ceil(R/block_rows), ceil(C/128)])."""
    x = _bits(x).contiguous()
    B, R, C = (1, *x.shape) if x.dim() == 2 else tuple(x.shape)
    q = torch.empty(x.shape, dtype=torch.uint8, device=x.device) if q is None else q
    nr, nc = -(-R // block_rows), -(-C // 128)
    scale = torch.empty((B, nr, nc), dtype=torch.float32, device=x.device) if scale is None else scale
    _lib.check("quantize_blockwise", _lib.lib().quantize_blockwise(_ptr(x), B, R, C, block_rows, codec, _ptr(q),
                                                                    _ptr(scale), _stream(stream)))
    return q, scale


def grouped_mm_blockwise(a, a_scale, b, b_scale, offs, n_groups, M, N, K, out=None, out_dtype=OUT_BF16, stream=None):
    """GROUPED_M over blockwise e4m3fn operands -> out [M, N] (bf16 or f32)."""
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16 if out_dtype == OUT_BF16 else torch.float32, device=a.device)
    _lib.check("grouped_mm_blockwise", _lib.lib().grouped_mm_blockwise(
        _ptr(a), OPD_E4M3FN, _ptr(a_scale), _ptr(b), OPD_E4M3FN, _ptr(b_scale), _ptr(offs), n_groups, M, N, K,
        _ptr(out), out_dtype, _stream(stream)))
    return out


def quantize_blockwise_tokens(x, offs, codec=E4M3FN, ld_q=None, q_t=None, scale=None, stream=None):
    """x bf16 [M, C], offs int32 [E] -> (q_t u8 [C, ld_q], scale f32 [block bound, C])."""
    x = _bits(x).contiguous()
    M, C = x.shape
    E = offs.numel()
    ld_q = (M + 15) // 16 * 16 if ld_q is None else ld_q
    q_t = torch.empty((C, ld_q), dtype=torch.uint8, device=x.device) if q_t is None else q_t
    nb = int(_lib.lib().blockwise_token_blocks_bound(M, E))
    scale = torch.empty((nb, C), dtype=torch.float32, device=x.device) if scale is None else scale
    _lib.check("quantize_blockwise_tokens", _lib.lib().quantize_blockwise_tokens(
        _ptr(x), M, C, _ptr(offs), E, codec, _ptr(q_t), ld_q, _ptr(scale), _stream(stream)))
    return q_t, scale


def grouped_mm_blockwise_k(a_t, a_scale, b_t, b_scale, offs, tokens, out=None, out_dtype=OUT_BF16, stream=None):
    """GROUPED_K over blockwise operands a_t [N, ld], b_t [K, ld] -> out [E, N, K]."""
    N, ld = a_t.shape
    K = b_t.shape[0]
    E = offs.numel()
    if out is None:
        out = torch.empty((E, N, K), dtype=torch.bfloat16 if out_dtype == OUT_BF16 else torch.float32,
                          device=a_t.device)
    _lib.check("grouped_mm_blockwise_k", _lib.lib().grouped_mm_blockwise_k(
        _ptr(a_t), _ptr(a_scale), _ptr(b_t), _ptr(b_scale), _ptr(offs), E, tokens, ld, N, K, _ptr(out), out_dtype,
        _stream(stream)))
    return out


def moe_route_rows_bound(slots: int, n_experts: int, pad: int = 1) -> int:
    return int(_lib.lib().moe_route_rows_bound(slots, n_experts, pad))


def moe_route_workspace_bytes(slots: int, n_experts: int) -> int:
    return int(_lib.lib().moe_route_workspace_bytes(slots, n_experts))


def moe_route(expert_ids, n_experts, pad=1, out=None, workspace=None, stream=None):
    """expert_ids int32 [T, k] -> (counts [E], offs [E], dest [T*k], src [rows bound]), all int32."""
    ids = expert_ids.contiguous()
    if ids.dtype != torch.int32 or ids.dim() != 2:
        raise ValueError("moe_route needs int32 expert ids of shape [tokens, topk]")
    T, k = ids.shape
    rows = moe_route_rows_bound(T * k, n_experts, pad)
    ws = int(_lib.lib().moe_route_workspace_bytes(T * k, n_experts))
    if rows < 0 or ws < 0:
        raise ValueError(f"moe_route: invalid sizes tokens={T} topk={k} experts={n_experts} pad={pad}")
    dev = ids.device
    if out is None:
        out = (torch.empty(n_experts, dtype=torch.int32, device=dev), torch.empty(n_experts, dtype=torch.int32, device=dev),
               torch.empty(T * k, dtype=torch.int32, device=dev), torch.empty(rows, dtype=torch.int32, device=dev))
    counts, offs, dest, src = out
    if workspace is None:
        workspace = torch.empty(max(ws, 4), dtype=torch.uint8, device=dev)
    _lib.check("moe_route", _lib.lib().moe_route(_ptr(ids), T, k, n_experts, pad, _ptr(counts), _ptr(offs),
                                                  _ptr(dest), _ptr(src), _ptr(workspace), _stream(stream)))
    return counts, offs, dest, src


def moe_route_noalloc(expert_ids, n_experts, out, pad=1, stream=None):
    """moe_route on the library's fixed scratch: nothing is allocated, so the outputs
    out = (counts [E], offs [E], dest [T*k], src [rows bound]) (int32) must be passed."""
    ids = expert_ids
    if ids.dtype != torch.int32 or ids.dim() != 2 or not ids.is_contiguous():
        raise ValueError("moe_route_noalloc needs contiguous int32 expert ids of shape [tokens, topk]")
    T, k = ids.shape
    counts, offs, dest, src = out
    _lib.check("moe_route_noalloc", _lib.lib().moe_route_noalloc(_ptr(ids), T, k, n_experts, pad, _ptr(counts),
                                                                  _ptr(offs), _ptr(dest), _ptr(src), _stream(stream)))
    return counts, offs, dest, src


def moe_permute(x, src, topk, xg=None, stream=None):
    """x bf16 [T, C], src int32 [R] -> xg bf16 [R, C]: row r = x[src[r] // topk], zeros where src[r] < 0."""
    x = _bits(x).contiguous()
    T, C = x.shape
    R = src.numel()
    xg = torch.empty((R, C), dtype=x.dtype, device=x.device) if xg is None else xg
    _lib.check("moe_permute", _lib.lib().moe_permute(_ptr(x), T, C, topk, _ptr(src), R, _ptr(xg), _stream(stream)))
    return xg


def moe_permute_quantized(q, scale, src, topk, codec=E4M3FN, qg=None, scale_g=None, stream=None):
    """Rowwise codes q u8 [T, C] and scales f32 [T], src int32 [R] -> (qg u8 [R, C], scale_g f32 [R])."""
    q = q.contiguous()
    T, C = q.shape
    R = src.numel()
    qg = torch.empty((R, C), dtype=_codes(codec), device=q.device) if qg is None else qg
    scale_g = torch.empty((R,), dtype=torch.float32, device=q.device) if scale_g is None else scale_g
    _lib.check("moe_permute_quantized", _lib.lib().moe_permute_quantized(
        _ptr(q), _ptr(scale), T, C, topk, _ptr(src), R, codec, _ptr(qg), _ptr(scale_g), _stream(stream)))
    return qg, scale_g


def moe_combine(yg, dest, weights, topk, y=None, stream=None):
    """yg bf16 [R, C], dest int32 [T*k], weights f32 [T, k] or None (every weight 1) -> y bf16 [T, C]."""
    yg = _bits(yg).contiguous()
    R, C = yg.shape
    T = dest.numel() // topk
    if weights is not None:
        weights = weights.contiguous()
        if weights.dtype != torch.float32 or tuple(weights.shape) != (T, topk):
            raise ValueError("moe_combine: weights f32 [T, topk]")
    if dest.numel() != T * topk:
        raise ValueError("moe_combine: dest [T*topk]")
    y = torch.empty((T, C), dtype=yg.dtype, device=yg.device) if y is None else y
    _lib.check("moe_combine", _lib.lib().moe_combine(_ptr(yg), R, _ptr(dest), _ptr(weights), T, topk, C, _ptr(y),
                                                     _stream(stream)))
    return y


def moe_permute_rowwise(x, src, topk, codec=E4M3FN, xg=None, qg=None, scale_g=None, keep_bf16=True, stream=None):
    """x bf16 [T, C], src int32 [R] -> (xg bf16 [R, C] or None, qg u8 [R, C], scale_g f32 [R]): the gathered
    rows and their rowwise codes in one pass (keep_bf16=False skips the bf16 copy)."""
    x = _bits(x).contiguous()
    T, C = x.shape
    R = src.numel()
    if keep_bf16:
        xg = torch.empty((R, C), dtype=x.dtype, device=x.device) if xg is None else xg
    else:
        xg = None
    qg = torch.empty((R, C), dtype=_codes(codec), device=x.device) if qg is None else qg
    scale_g = torch.empty((R,), dtype=torch.float32, device=x.device) if scale_g is None else scale_g
    _lib.check("moe_permute_rowwise", _lib.lib().moe_permute_rowwise(
        _ptr(x), T, C, topk, _ptr(src), R, codec, _ptr(xg), _ptr(qg), _ptr(scale_g), _stream(stream)))
    return xg, qg, scale_g


def moe_combine_backward(dy, yg, dest, src, weights, topk, codec=E4M3FN, codes=True, dyg=None, q=None, scale=None,
                         dweights=None, stream=None, rows_out=True):
    """dy bf16 [T, C], yg bf16 [R, C], dest int32 [T*k], src int32 [R], weights f32 [T, k] ->
    (dyg bf16 [R, C] or None, q u8 [R, C] or None, scale f32 [R] or None, dweights f32 [T*k]).
    rows_out=False: the routed-row gradients are not written (dyg is None)."""
    dy = _bits(dy).contiguous()
    yg = _bits(yg).contiguous()
    T, C = dy.shape
    R = yg.shape[0]
    weights = weights.contiguous()
    if weights.dtype != torch.float32 or tuple(weights.shape) != (T, topk) or dest.numel() != T * topk \
            or src.numel() != R or yg.shape[1] != C:
        raise ValueError("moe_combine_backward: dy [T, C], yg [R, C], weights f32 [T, topk], dest [T*topk], src [R]")
    dev = dy.device
    if rows_out:
        dyg = torch.empty((R, C), dtype=dy.dtype, device=dev) if dyg is None else dyg
    else:
        dyg = None
    if codes:
        q = torch.empty((R, C), dtype=torch.uint8, device=dev) if q is None else q
        scale = torch.empty((R,), dtype=torch.float32, device=dev) if scale is None else scale
    else:
        q = scale = None
    dweights = torch.empty((T * topk,), dtype=torch.float32, device=dev) if dweights is None else dweights
    _lib.check("moe_combine_backward", _lib.lib().moe_combine_backward(
        _ptr(dy), _ptr(yg), R, _ptr(dest), _ptr(src), _ptr(weights), T, topk, C, codec, _ptr(dyg), _ptr(q),
        _ptr(scale), _ptr(dweights), _stream(stream)))
    return dyg, q, scale, dweights


_HERE = contextlib.nullcontext()


def _on(fn, stream, first, *others):
    """The context an operator allocates and launches in: the device of its tensors (all on one GPU) and the given
    stream, so that temporary and output memory belongs to the stream that uses it."""
    at = first.get_device()
    for t in others:
        if t is not None and t.get_device() != at:
            raise ValueError(f"{fn}: tensors on {first.device} and {t.device}")
    if at < 0:
        raise ValueError(f"{fn}: needs GPU tensors, got {first.device}")
    if stream is not None:
        if stream.device != first.device:
            raise ValueError(f"{fn}: tensors on {first.device}, stream on {stream.device}")
        return torch.cuda.stream(stream)
    return _HERE if at == torch.cuda.current_device() else torch.cuda.device(at)


def _current(t):
    """The raw handle of the current stream on t's device (torch.cuda.current_stream builds a Stream object first: 2.8 us
    instead of 0.1, a fifth of a small call)."""
    return torch._C._cuda_getCurrentRawStream(t.get_device())


def _rows2d(fn, name, t, dtypes):
    """(rows, cols, row stride) of a 2D tensor whose rows are contiguous; other strides are refused, not copied."""
    if t.dim() != 2 or t.dtype not in dtypes:
        raise ValueError(f"{fn}: {name} must be a 2D tensor of {' or '.join(map(str, dtypes))}, got {t.dtype} "
                         f"{tuple(t.shape)}")
    R, C = t.shape
    if R == 0 or C == 0:
        return R, C, C
    ld, step = t.stride()
    if (step != 1 and C > 1) or (ld < C and R > 1):
        raise ValueError(f"{fn}: {name} needs contiguous rows that do not overlap, got strides {t.stride()}")
    return R, C, ld if R > 1 else C


def _out(fn, name, t, shape, dtype, dev):
    """A caller's output tensor, checked, or a new one."""
    if t is None:   # spelt out for its size: 1.3 us instead of torch.empty's 1.7, five times in a small norm call
        if len(shape) == 2:
            return torch.empty_strided(shape, (shape[1], 1), dtype=dtype, device=dev)
        return torch.empty(shape, dtype=dtype, device=dev)
    if t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous() or t.device != dev:
        raise ValueError(f"{fn}: {name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {dev}, got "
                         f"{t.dtype} {tuple(t.shape)} on {t.device}")
    return t


def _given(fn, name, t, shape, dtypes, dev):
    """A caller's output tensor is None or has this shape, one of these types and this device, contiguous."""
    if t is not None and (t.dtype not in dtypes or tuple(t.shape) != tuple(shape) or not t.is_contiguous() or t.device != dev):
        raise ValueError(f"{fn}: {name} must be a contiguous {' or '.join(map(str, dtypes))} tensor of shape {tuple(shape)} on "
                         f"{dev}, got {t.dtype} {tuple(t.shape)} on {t.device}")


def _vec(fn, name, t, n, dtypes):
    if t is not None and (t.dtype not in dtypes or t.dim() != 1 or t.numel() != n or not t.is_contiguous()):
        raise ValueError(f"{fn}: {name} must be a contiguous {' or '.join(map(str, dtypes))} tensor of {n} elements, "
                         f"got {t.dtype} {tuple(t.shape)}")


def _workspace(fn, workspace, need, dev):
    """A caller's workspace, checked, or a new one."""
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=dev)
    if (workspace.numel() * workspace.element_size() < need or not workspace.is_contiguous() or
            workspace.device != dev):
        raise ValueError(f"{fn}: a contiguous workspace of {need} bytes needed on {dev}")
    return workspace


_BF16, _F32, _I32, _U8 = (torch.bfloat16,), (torch.float32,), (torch.int32,), (torch.uint8,)
_BF16_F32 = (torch.bfloat16, torch.float32)


def _norm_inputs(fn, x, gamma, residual):
    R, C, ld = _rows2d(fn, "x", x, _BF16)
    ld_r = C
    if residual is not None:
        Rr, Cr, ld_r = _rows2d(fn, "residual", residual, _BF16)
        if (Rr, Cr) != (R, C):
            raise ValueError(f"{fn}: residual must have x's shape {(R, C)}, got {(Rr, Cr)}")
    _vec(fn, "gamma", gamma, C, _BF16_F32)
    return R, C, ld, ld_r, OUT_BF16 if gamma is not None and gamma.dtype == torch.bfloat16 else OUT_F32


def rmsnorm_quantize_rowwise(x, gamma=None, eps=1e-6, residual=None, codec=E4M3FN, keep_bf16=True, codes=True,
                             sum_out=None, h=None, q=None, scale=None, rstd=None, stream=None):
    """x bf16 [R, C] (row stride may exceed C), gamma bf16 or f32 [C] or None, residual bf16 [R, C] or None ->
    (h bf16 [R, C] or None, q u8 [R, C] or None, scale f32 [R] or None, rstd f32 [R], sum bf16 [R, C]): the residual's
    addition, the RMS norm and the rowwise quantization of the normed rows (from fp32; int8 codes with codec=INT8) in one
    pass.  sum is x + residual, the new residual stream (x itself without a residual); sum_out may be x or residual (contiguous).
    keep_bf16=False skips h, codes=False skips q and scale."""
    fn = "rmsnorm_quantize_rowwise"
    R, C, ld, ld_r, gt = _norm_inputs(fn, x, gamma, residual)
    with _on(fn, stream, x, gamma, residual):
        dev = x.device
        s = _out(fn, "sum_out", sum_out, (R, C), torch.bfloat16, dev) if residual is not None else x
        h = _out(fn, "h", h, (R, C), torch.bfloat16, dev) if keep_bf16 else None
        q = _out(fn, "q", q, (R, C), _codes(codec), dev) if codes else None
        scale = _out(fn, "scale", scale, (R,), torch.float32, dev) if codes else None
        rstd = _out(fn, "rstd", rstd, (R,), torch.float32, dev)
        _lib.check(fn, _lib.lib().rmsnorm_quantize_rowwise(
            _ptr(x), _ptr(residual), _ptr(gamma), gt, R, C, ld, ld_r, eps, codec, _ptr(s), _ptr(h), _ptr(q),
            _ptr(scale), _ptr(rstd), _current(x)))
    return h, q, scale, rstd, s


def rmsnorm_quantize_mx(x, gamma=None, eps=1e-6, residual=None, rule=MX_FLOOR_OCP, layout=MX_LAYOUT_ROWS, keep_bf16=True,
                        sum_out=None, h=None, q=None, scale=None, rstd=None, stream=None):
    """As rmsnorm_quantize_rowwise with MXFP8 codes: scale is e8m0 u8 [R, C / 32], or of shape
    mx_k4_shape(R, C // 32) with layout=MX_LAYOUT_K4."""
    fn = "rmsnorm_quantize_mx"
    R, C, ld, ld_r, gt = _norm_inputs(fn, x, gamma, residual)
    with _on(fn, stream, x, gamma, residual):
        dev = x.device
        s = _out(fn, "sum_out", sum_out, (R, C), torch.bfloat16, dev) if residual is not None else x
        h = _out(fn, "h", h, (R, C), torch.bfloat16, dev) if keep_bf16 else None
        q = _out(fn, "q", q, (R, C), torch.uint8, dev)
        scale = _out(fn, "scale", scale, mx_k4_shape(R, C // 32) if layout == MX_LAYOUT_K4 else (R, C // 32), torch.uint8,
                     dev)
        rstd = _out(fn, "rstd", rstd, (R,), torch.float32, dev)
        _lib.check(fn, _lib.lib().rmsnorm_quantize_mx(
            _ptr(x), _ptr(residual), _ptr(gamma), gt, R, C, ld, ld_r, eps, rule, layout, _ptr(s), _ptr(h), _ptr(q),
            _ptr(scale), _ptr(rstd), _current(x)))
    return h, q, scale, rstd, s


def rmsnorm_backward_workspace_bytes(rows: int, cols: int) -> int:
    return int(_lib.lib().rmsnorm_backward_workspace_bytes(rows, cols))


def rmsnorm_backward(dh, s, rstd, gamma=None, dsum=None, dx=None, dgamma=None, want_dgamma=True, workspace=None,
                     stream=None):
    """dh bf16 [R, C] (the gradient of h), s bf16 [R, C] and rstd f32 [R] from the forward (s = x without a residual),
    gamma as there, dsum bf16 [R, C] or None (the gradient that reaches the residual stream past the norm) ->
    (dx bf16 [R, C], the gradient of x and of the residual, dgamma f32 [C] or None).  dx may be dh, s or dsum.  dh, s and
    dsum are contiguous: an x whose rows lie further apart is refused here, not copied."""
    fn = "rmsnorm_backward"
    dims = []
    for name, t in (("dh", dh), ("s", s), ("dsum", dsum)):
        if t is not None:
            R, C, ld = _rows2d(fn, name, t, _BF16)
            if ld != C and R > 1:
                raise ValueError(f"{fn}: {name} must be contiguous, got strides {t.stride()}")
            dims.append((R, C))
    if len(set(dims)) != 1:
        raise ValueError(f"{fn}: dh, s and dsum must have one shape, got {dims}")
    R, C = dims[0]
    _vec(fn, "rstd", rstd, R, _F32)
    _vec(fn, "gamma", gamma, C, _BF16_F32)
    with _on(fn, stream, dh, s, rstd, gamma, dsum, workspace):
        dev = dh.device
        dx = _out(fn, "dx", dx, (R, C), torch.bfloat16, dev)
        dgamma = _out(fn, "dgamma", dgamma, (C,), torch.float32, dev) if want_dgamma else None
        if want_dgamma:
            workspace = _workspace(fn, workspace, max(rmsnorm_backward_workspace_bytes(R, C), 16), dev)
        _lib.check(fn, _lib.lib().rmsnorm_backward(
            _ptr(dh), _ptr(s), _ptr(rstd), _ptr(gamma),
            OUT_BF16 if gamma is not None and gamma.dtype == torch.bfloat16 else OUT_F32, _ptr(dsum), R, C, _ptr(dx),
            _ptr(dgamma), _ptr(workspace) if want_dgamma else None, _current(dh)))
    return dx, dgamma


def _gate_inputs(fn, logits, token_mask):
    T, E, ld = _rows2d(fn, "logits", logits, _BF16_F32)
    if not 1 <= E < 2**31:   # an int32 argument
        raise ValueError(f"{fn}: logits need at least one expert, fewer than 2^31, got {E}")
    _vec(fn, "token_mask", token_mask, T, (torch.uint8, torch.bool))
    return T, E, ld, OUT_F32 if logits.dtype == torch.float32 else OUT_BF16


def _gate_topk(fn, topk, E):
    if not 1 <= topk <= E:
        raise ValueError(f"{fn}: topk must be between 1 and the {E} experts, got {topk}")


def _gate_slots(fn, name, t, T, dtypes):
    """topk of a contiguous [T, topk] tensor of slots."""
    if t.dim() != 2 or t.shape[0] != T or t.dtype not in dtypes or not t.is_contiguous():
        raise ValueError(f"{fn}: {name} must be a contiguous {dtypes[0]} tensor of shape [{T}, topk], got {t.dtype} "
                         f"{tuple(t.shape)}")
    return t.shape[1]


def _gate_seqs(fn, seq_offs):
    if seq_offs is None:
        return 1
    if not 1 <= seq_offs.numel() < 2**31:   # an int32 argument
        raise ValueError(f"{fn}: seq_offs needs at least one sequence, fewer than 2^31, got {seq_offs.numel()}")
    _vec(fn, "seq_offs", seq_offs, seq_offs.numel(), _I32)
    return seq_offs.numel()


def moe_gate(logits, topk, score=GATE_SOFTMAX, bias=None, token_mask=None, renormalize=False, route_scale=1.0, ids=None,
             weights=None, stream=None):
    """logits f32 or bf16 [T, E] (row stride may exceed E), bias f32 [E] or None (added for the choice only), token_mask
    u8 or bool [T] or None -> (ids int32 [T, topk], weights f32 [T, topk]): each token's topk experts in decreasing
    order (ties to the lower index; -1 with weight 0 where no eligible expert is left) and their weights, what
    moe_route and moe_combine take."""
    fn = "moe_gate"
    T, E, ld, dt = _gate_inputs(fn, logits, token_mask)
    _gate_topk(fn, topk, E)
    _vec(fn, "bias", bias, E, _F32)
    with _on(fn, stream, logits, bias, token_mask):
        ids = _out(fn, "ids", ids, (T, topk), torch.int32, logits.device)
        weights = _out(fn, "weights", weights, (T, topk), torch.float32, logits.device)
        _lib.check(fn, _lib.lib().moe_gate(_ptr(logits), dt, T, E, ld, topk, score, _ptr(bias), _ptr(token_mask),
                                           bool(renormalize), route_scale, _ptr(ids), _ptr(weights), _current(logits)))
    return ids, weights


def moe_balance_workspace_bytes(tokens: int, n_experts: int, n_seqs: int = 1) -> int:
    return int(_lib.lib().moe_balance_workspace_bytes(tokens, n_experts, n_seqs))


def _balance_outputs(fn, T, E, S, loss, counts, dprob, workspace, dev):
    need = moe_balance_workspace_bytes(T, E, S)
    if need < 0:
        raise ValueError(f"{fn}: invalid sizes tokens={T} experts={E} sequences={S}")
    workspace = _workspace(fn, workspace, need, dev)
    return (_out(fn, "loss", loss, (1,), torch.float32, dev), _out(fn, "counts", counts, (S, E), torch.int32, dev),
            _out(fn, "dprob", dprob, (S, E), torch.float32, dev), workspace)


def moe_gate_balance(logits, topk, coef, seq_offs=None, score=GATE_SOFTMAX, bias=None, token_mask=None,
                     renormalize=False, route_scale=1.0, ids=None, weights=None, loss=None, counts=None, dprob=None,
                     workspace=None, stream=None):
    """moe_gate and moe_balance_loss of its choices from one read of the logits -> (ids, weights, loss f32 [1], counts
    int32 [S, E], dprob f32 [S, E]); seq_offs int32 [S] are the inclusive ends of the sequences (None: one of all tokens)."""
    fn = "moe_gate_balance"
    T, E, ld, dt = _gate_inputs(fn, logits, token_mask)
    _gate_topk(fn, topk, E)
    _vec(fn, "bias", bias, E, _F32)
    S = _gate_seqs(fn, seq_offs)
    with _on(fn, stream, logits, bias, token_mask, seq_offs):
        dev = logits.device
        ids = _out(fn, "ids", ids, (T, topk), torch.int32, dev)
        weights = _out(fn, "weights", weights, (T, topk), torch.float32, dev)
        loss, counts, dprob, workspace = _balance_outputs(fn, T, E, S, loss, counts, dprob, workspace, dev)
        _lib.check(fn, _lib.lib().moe_gate_balance(
            _ptr(logits), dt, T, E, ld, topk, score, _ptr(bias), _ptr(token_mask), bool(renormalize), route_scale,
            _ptr(ids), _ptr(weights), _ptr(seq_offs), S, coef, _ptr(loss), _ptr(counts), _ptr(dprob), _ptr(workspace),
            _current(logits)))
    return ids, weights, loss, counts, dprob


def moe_balance_loss(logits, ids, coef, seq_offs=None, score=GATE_SOFTMAX, token_mask=None, loss=None, counts=None,
                     dprob=None, workspace=None, stream=None):
    """logits f32 or bf16 [T, E], ids int32 [T, topk] -> (loss f32 [1], counts int32 [S, E], dprob f32 [S, E]): the
    load-balance loss of the choices, how many slots of each sequence chose each expert, and what the backward takes."""
    fn = "moe_balance_loss"
    T, E, ld, dt = _gate_inputs(fn, logits, token_mask)
    topk = _gate_slots(fn, "ids", ids, T, _I32)
    _gate_topk(fn, topk, E)
    S = _gate_seqs(fn, seq_offs)
    with _on(fn, stream, logits, ids, token_mask, seq_offs):
        loss, counts, dprob, workspace = _balance_outputs(fn, T, E, S, loss, counts, dprob, workspace, logits.device)
        _lib.check(fn, _lib.lib().moe_balance_loss(
            _ptr(logits), dt, T, E, ld, topk, score, _ptr(token_mask), _ptr(ids), _ptr(seq_offs), S, coef, _ptr(loss),
            _ptr(counts), _ptr(dprob), _ptr(workspace), _current(logits)))
    return loss, counts, dprob


def moe_gate_backward(logits, ids, dweights, score=GATE_SOFTMAX, token_mask=None, renormalize=False, route_scale=1.0,
                      dprob=None, dloss=None, seq_offs=None, dlogits=None, stream=None):
    """The gradient [T, E] of the logits (in their type) for dweights f32 [T, topk] (or flat, as moe_combine_backward
    gives it) and, with dprob f32 [S, E] from the forward, for the balance loss (dloss f32 [1] on the device, None: 1)."""
    fn = "moe_gate_backward"
    T, E, ld, dt = _gate_inputs(fn, logits, token_mask)
    topk = _gate_slots(fn, "ids", ids, T, _I32)
    _gate_topk(fn, topk, E)
    if dweights.dim() == 1 and dweights.numel() == T * topk:
        dweights = dweights.view(T, topk)
    if _gate_slots(fn, "dweights", dweights, T, _F32) != topk:
        raise ValueError(f"{fn}: dweights must have ids' shape {(T, topk)}, got {tuple(dweights.shape)}")
    return _gate_backward(fn, logits, T, E, ld, dt, topk, ids, dweights, score, token_mask, renormalize, route_scale, dprob,
                          dloss, seq_offs, dlogits, stream)


def moe_balance_loss_backward(logits, dprob, dloss=None, seq_offs=None, score=GATE_SOFTMAX, token_mask=None,
                              dlogits=None, stream=None):
    """The gradient [T, E] of the logits (in their type) through the balance loss alone."""
    fn = "moe_balance_loss_backward"
    T, E, ld, dt = _gate_inputs(fn, logits, token_mask)
    if dprob is None:
        raise ValueError(f"{fn}: needs dprob")
    return _gate_backward(fn, logits, T, E, ld, dt, 1, None, None, score, token_mask, False, 1.0, dprob, dloss, seq_offs,
                          dlogits, stream)


def _gate_backward(fn, logits, T, E, ld, dt, topk, ids, dweights, score, token_mask, renormalize, route_scale, dprob,
                   dloss, seq_offs, dlogits, stream):
    S = _gate_seqs(fn, seq_offs)
    if dprob is None and (dloss is not None or seq_offs is not None):
        raise ValueError(f"{fn}: dloss and seq_offs go with dprob")
    if dprob is not None and (dprob.dtype != torch.float32 or tuple(dprob.shape) != (S, E) or not dprob.is_contiguous()):
        raise ValueError(f"{fn}: dprob must be a contiguous torch.float32 tensor of shape {(S, E)}, got {dprob.dtype} "
                         f"{tuple(dprob.shape)}")
    if dloss is not None and (dloss.dtype != torch.float32 or dloss.numel() != 1):
        raise ValueError(f"{fn}: dloss must be one torch.float32 value on the device")
    with _on(fn, stream, logits, ids, dweights, token_mask, dprob, dloss, seq_offs):
        dlogits = _out(fn, "dlogits", dlogits, (T, E), logits.dtype, logits.device)
        _lib.check(fn, _lib.lib().moe_gate_backward(
            _ptr(logits), dt, T, E, ld, topk, score, _ptr(token_mask), bool(renormalize), route_scale, _ptr(ids),
            _ptr(dweights), _ptr(seq_offs), S, _ptr(dprob), _ptr(dloss), _ptr(dlogits), _current(logits)))
    return dlogits


_F8_CODES = (torch.uint8, torch.float8_e4m3fn)
_E8M0_CODES = (torch.uint8, torch.float8_e8m0fnu)


def _saved_input(fn, hq, hs):
    """(rows, F) of a SwiGLU input kept in MXFP8 [R, 2F] with row-major scales [R, 2F / 32]."""
    R, F2, ld = _rows2d(fn, "hq", hq, _F8_CODES)
    if F2 % 64 or (ld != F2 and R > 1):
        raise ValueError(f"{fn}: hq must be contiguous [R, 2F] with F a multiple of 32, got {tuple(hq.shape)}, strides {hq.stride()}")
    if hs.dtype not in _E8M0_CODES or tuple(hs.shape) != (R, F2 // 32) or not hs.is_contiguous():
        raise ValueError(f"{fn}: hs must be a contiguous e8m0 (uint8) tensor of shape {(R, F2 // 32)}, got {hs.dtype} "
                         f"{tuple(hs.shape)}")
    return R, F2 // 2


def _saved_gradient(fn, da2, R, F):
    if tuple(da2.shape) != (R, F) or da2.dtype != torch.bfloat16 or not da2.is_contiguous():
        raise ValueError(f"{fn}: da2 must be a contiguous torch.bfloat16 tensor of shape {(R, F)}, got {da2.dtype} "
                         f"{tuple(da2.shape)}")


def swiglu_quantize_rowwise_save(h1, codec=E4M3FN, rule=MX_FLOOR_OCP, keep_bf16=False, a2=None, q=None, scale=None,
                                 hq=None, hs=None, stream=None):
    """h1 bf16 [R, 2F] (gate | up; row stride may exceed 2F) -> (a2 bf16 [R, F] or None, q u8 [R, F], scale f32 [R], hq u8
    [R, 2F], hs u8 [R, 2F / 32]): the rowwise codes of silu(gate) * up (from fp32) for the W2 product, and h1 in MXFP8, all
    that the backward needs of it.  keep_bf16=True also writes bf16(silu(gate) * up)."""
    fn = "swiglu_quantize_rowwise_save"
    R, F2, ld = _rows2d(fn, "h1", h1, _BF16)
    if F2 % 64:
        raise ValueError(f"{fn}: h1 needs 2F columns with F a multiple of 32, got {F2}")
    F = F2 // 2
    with _on(fn, stream, h1):
        dev = h1.device
        a2 = _out(fn, "a2", a2, (R, F), torch.bfloat16, dev) if keep_bf16 else None
        q = _out(fn, "q", q, (R, F), torch.uint8, dev)
        scale = _out(fn, "scale", scale, (R,), torch.float32, dev)
        hq = _out(fn, "hq", hq, (R, F2), torch.uint8, dev)
        hs = _out(fn, "hs", hs, (R, F2 // 32), torch.uint8, dev)
        _lib.check(fn, _lib.lib().swiglu_quantize_rowwise_save(
            _ptr(h1), R, F, ld, codec, rule, _ptr(a2), _ptr(q), _ptr(scale), _ptr(hq), _ptr(hs), _current(h1)))
    return a2, q, scale, hq, hs


def swiglu_backward_quantize_rowwise_saved(da2, hq, hs, codec=E4M3FN, keep_bf16=True, codes=True, want_a2=False, dh1=None,
                                           q=None, scale=None, a2=None, stream=None):
    """da2 bf16 [R, F] and the input kept in MXFP8, hq [R, 2F] and hs [R, 2F / 32] -> (dh1 bf16 [R, 2F] or None, q u8 [R, 2F]
    or None, scale f32 [R] or None, a2 bf16 [R, F] or None): SwiGLU's input gradient and its rowwise codes (from fp32), and
    with want_a2 the activation again.  keep_bf16=False skips dh1, codes=False skips q and scale."""
    fn = "swiglu_backward_quantize_rowwise_saved"
    R, F = _saved_input(fn, hq, hs)
    _saved_gradient(fn, da2, R, F)
    if not (keep_bf16 or codes or want_a2):
        raise ValueError(f"{fn}: no result asked for")
    with _on(fn, stream, da2, hq, hs):
        dev = da2.device
        dh1 = _out(fn, "dh1", dh1, (R, 2 * F), torch.bfloat16, dev) if keep_bf16 else None
        q = _out(fn, "q", q, (R, 2 * F), torch.uint8, dev) if codes else None
        scale = _out(fn, "scale", scale, (R,), torch.float32, dev) if codes else None
        a2 = _out(fn, "a2", a2, (R, F), torch.bfloat16, dev) if want_a2 else None
        _lib.check(fn, _lib.lib().swiglu_backward_quantize_rowwise_saved(
            _ptr(da2), _ptr(hq), _ptr(hs), R, F, codec, _ptr(dh1), _ptr(q), _ptr(scale), _ptr(a2), _current(da2)))
    return dh1, q, scale, a2


def _saved_groups(fn, offs):
    if offs.numel() < 1:
        raise ValueError(f"{fn}: offs needs at least one group")
    _vec(fn, "offs", offs, offs.numel(), _I32)


def _given_dual_outputs(fn, R, C, offs, rows_pad, layout, dev, bf16_name, bf16, q, scale, q_t, scale_t, offs_pad):
    """Checks the caller's outputs of a dual form of R rows of C columns."""
    rp = rows_pad or quantize_mx_rows_bound(R, offs.numel())
    sc_shape = mx_k4_shape if layout == MX_LAYOUT_K4 else lambda n_rows, n_blocks: (n_rows, n_blocks)
    _given(fn, bf16_name, bf16, (R, C), _BF16, dev)
    _given(fn, "q", q, (R, C), _F8_CODES, dev)
    _given(fn, "scale", scale, sc_shape(R, C // 32), _E8M0_CODES, dev)
    _given(fn, "q_t", q_t, (C, rp), _F8_CODES, dev)
    _given(fn, "scale_t", scale_t, sc_shape(C, rp // 32), _E8M0_CODES, dev)
    _given(fn, "offs_pad", offs_pad, (offs.numel(),), _I32, dev)


def swiglu_quantize_mx_dual_saved(hq, hs, offs, rule=MX_FLOOR_OCP, rows_pad=None, a2=None, q=None, scale=None, q_t=None,
                                  scale_t=None, offs_pad=None, layout=MX_LAYOUT_K4, stream=None):
    """swiglu_quantize_mx_dual from the input kept in MXFP8, hq [R, 2F] and hs [R, 2F / 32]: the same results from the kept
    values (the W2 weight gradient's operand, formed again in the backward)."""
    fn = "swiglu_quantize_mx_dual_saved"
    R, F = _saved_input(fn, hq, hs)
    _saved_groups(fn, offs)
    _given_dual_outputs(fn, R, F, offs, rows_pad, layout, hq.device, "a2", a2, q, scale, q_t, scale_t, offs_pad)
    with _on(fn, stream, hq, hs, offs):
        rp, q, scale, q_t, scale_t, offs_pad = _mx_dual_outputs(R, F, offs, rows_pad, q, scale, q_t, scale_t, offs_pad,
                                                                layout, hq.device)
        _lib.check(fn, _lib.lib().swiglu_quantize_mx_dual_saved(
            _ptr(hq), _ptr(hs), R, F, _ptr(offs), offs.numel(), rule, layout, _ptr(a2), _ptr(q), _ptr(scale), _ptr(q_t),
            _ptr(scale_t), rp, _ptr(offs_pad), _current(hq)))
    return a2, q, scale, q_t, scale_t, offs_pad


def swiglu_backward_quantize_mx_dual_saved(da2, hq, hs, offs, rule=MX_FLOOR_OCP, rows_pad=None, dh1=None, q=None,
                                           scale=None, q_t=None, scale_t=None, offs_pad=None, layout=MX_LAYOUT_K4,
                                           stream=None):
    """swiglu_backward_quantize_mx_dual from the input kept in MXFP8, hq [R, 2F] and hs [R, 2F / 32] (F a multiple of 128)."""
    fn = "swiglu_backward_quantize_mx_dual_saved"
    R, F = _saved_input(fn, hq, hs)
    _saved_gradient(fn, da2, R, F)
    _saved_groups(fn, offs)
    _given_dual_outputs(fn, R, 2 * F, offs, rows_pad, layout, hq.device, "dh1", dh1, q, scale, q_t, scale_t, offs_pad)
    with _on(fn, stream, da2, hq, hs, offs):
        rp, q, scale, q_t, scale_t, offs_pad = _mx_dual_outputs(R, 2 * F, offs, rows_pad, q, scale, q_t, scale_t, offs_pad,
                                                                layout, hq.device)
        _lib.check(fn, _lib.lib().swiglu_backward_quantize_mx_dual_saved(
            _ptr(da2), _ptr(hq), _ptr(hs), R, F, _ptr(offs), offs.numel(), rule, layout, _ptr(dh1), _ptr(q), _ptr(scale),
            _ptr(q_t), _ptr(scale_t), rp, _ptr(offs_pad), _current(da2)))
    return dh1, q, scale, q_t, scale_t, offs_pad


def moe_few_tokens_workspace_bytes(tokens: int, topk: int, cols: int, ffn: int) -> int:
    return int(_lib.lib().moe_few_tokens_workspace_bytes(tokens, topk, cols, ffn))


def _few_weights(fn, name, w, scale, E, rows, cols, w_fmt, scale_kind):
    """Quantized weights [E, rows, cols] of the given format and their scales, checked."""
    dtypes = (torch.int8, torch.uint8) if w_fmt == OPD_INT8 else (torch.uint8, torch.float8_e4m3fn)
    if tuple(w.shape) != (E, rows, cols) or w.dtype not in dtypes or not w.is_contiguous():
        raise ValueError(f"{fn}: {name} must be a contiguous {' or '.join(map(str, dtypes))} tensor of shape "
                         f"{(E, rows, cols)}, got {w.dtype} {tuple(w.shape)}")
    n = E * rows
    if scale_kind == SCALE_F32:
        dtypes, need = _F32, n
    else:
        nb = cols // 32
        dtypes, need = _E8M0_CODES, 4 * n * -(-nb // 4) if scale_kind == SCALE_E8M0_K4 else n * nb
    if scale.dtype not in dtypes or scale.numel() != need or not scale.is_contiguous():
        raise ValueError(f"{fn}: {name}_scale must be a contiguous {' or '.join(map(str, dtypes))} tensor of {need} elements, "
                         f"got {scale.dtype} {tuple(scale.shape)}")


def moe_few_tokens(x, ids, weights, w1, w1_scale, w2, w2_scale, w_fmt=OPD_E4M3FN, scale_kind=SCALE_F32, y=None,
                   workspace=None, stream=None):
    """The whole expert block for at most 64 tokens: x bf16 [T, K] (row stride may exceed K), ids int32 and weights f32
    [T, topk] (as moe_gate gives them), w1 [E, 2F, K] (gate | up rows) and w2 [E, K, F] in 8 bits with their scales ->
    y bf16 [T, K] = the weighted sum of the experts' SwiGLU blocks.  Formats: e4m3fn codes (uint8 or float8_e4m3fn) with
    f32 row scales or e8m0 scales (uint8 or float8_e8m0fnu; SCALE_E8M0, SCALE_E8M0_K4), or OPD_INT8 codes with f32 row
    scales, as quantize_rowwise and quantize_mx give them.  y may be x (contiguous)."""
    fn = "moe_few_tokens"
    T, K, ld = _rows2d(fn, "x", x, _BF16)
    topk = _gate_slots(fn, "ids", ids, T, _I32)
    if topk < 1 or _gate_slots(fn, "weights", weights, T, _F32) != topk:
        raise ValueError(f"{fn}: ids and weights must have one shape [T, topk], got {tuple(ids.shape)}, {tuple(weights.shape)}")
    if w1.dim() != 3 or w1.shape[1] % 2:
        raise ValueError(f"{fn}: w1 must have the shape [E, 2F, K], got {tuple(w1.shape)}")
    E, F = w1.shape[0], w1.shape[1] // 2
    _few_weights(fn, "w1", w1, w1_scale, E, 2 * F, K, w_fmt, scale_kind)
    _few_weights(fn, "w2", w2, w2_scale, E, K, F, w_fmt, scale_kind)
    with _on(fn, stream, x, ids, weights, w1, w1_scale, w2, w2_scale, workspace):
        dev = x.device
        y = _out(fn, "y", y, (T, K), torch.bfloat16, dev)
        workspace = _workspace(fn, workspace, max(moe_few_tokens_workspace_bytes(T, topk, K, F), 16), dev)
        _lib.check(fn, _lib.lib().moe_few_tokens(
            _ptr(x), T, K, ld, _ptr(ids), _ptr(weights), topk, _ptr(w1), _ptr(w1_scale), _ptr(w2), _ptr(w2_scale), w_fmt,
            scale_kind, E, F, _ptr(y), _ptr(workspace), _current(x)))
    return y


def encode_f32(y, codec=E4M3FN, q=None, stream=None):
    """The device FP8 encoder on fp32 values already inside [-fmax, fmax]."""
    q = torch.empty(y.shape, dtype=torch.uint8, device=y.device) if q is None else q
    _lib.check("fp8moe_encode_f32", _lib.lib().fp8moe_encode_f32(_ptr(y), y.numel(), codec, _ptr(q),
                                                                 _stream(stream)))
    return q


def default_codec(device: int = 0) -> int:
    import ctypes
    out = ctypes.c_int(-1)
    _lib.check("fp8moe_default_codec", _lib.lib().fp8moe_default_codec(device, ctypes.byref(out)))
    return out.value
