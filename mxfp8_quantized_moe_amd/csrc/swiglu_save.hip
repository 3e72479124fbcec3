// SwiGLU whose input is kept for the backward pass in 8 bits, and the backward
// that reads it, each fused with the rowwise FP8 quantization of its output.
//
// What is kept of h1 = [gate | up] is its MXFP8 form (e4m3fn codes, one e8m0 scale
// for 32 columns): 1.03 bytes a value instead of two, and the activation a2 = silu(gate) * up,
// two bytes more, need not be kept at all, since the backward forms it again from the same codes.
//
//   forward:   a = g s u, s = sigmoid(g): codes of a, the kept form of h1, bf16(a) if asked
//   backward:  with g, u the kept values and d the gradient of a,
//              d gate = d u s (1 + g (1 - s)),  d up = d g s:  bf16, their codes, and bf16(g s u) if asked
//
// The codes are cast from the fp32 results, not from their bf16 copies: one rounding
// instead of two.  The forward's own result does not depend on what is kept.
//
// A row stays in registers from the load to the cast: TPR threads own it, each with ITEMS chunks
// of eight columns; four neighbouring lanes hold one block of 32.  Rows beyond that are read twice and
// computed twice.
//
// 49152 x 1408: forward 86 us (5.7 TB/s of 7 bytes a value; the vector units issue all the time), backward with a2
// 141 us (5.9 TB/s; they issue 78% of it).
#include "device_common.hpp"
#include "kernels.hpp"
#include "swiglu_common.hpp"

namespace fp8moe {

typedef float sv_f32x2 __attribute__((ext_vector_type(2)));

struct SaveArgs {
  int64_t rows, F, ld_h1;
  const uint16_t* h1;     // forward
  const uint16_t* da2;    // backward
  uint8_t* hq;            // [rows][2F], written by the forward
  uint8_t* hs;            // [rows][2F / 32]
  int rule;
  uint8_t* q;             // codes of a [rows][F] (of dh1 [rows][2F]) or null
  float* scale;
  uint16_t* a2;           // [rows][F] or null
  uint16_t* dh1;          // [rows][2F] or null
};

template <int TPR>
__device__ __forceinline__ float sv_row_max(float m, float* red) {
  uint32_t v = __float_as_uint(m);   // magnitudes order as their patterns
  if constexpr (TPR <= 64) return __uint_as_float(group_max_u32<TPR>(v));
  v = group_max_u32<64>(v);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = __uint_as_float(v);
  __syncthreads();
  return fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
}

__device__ __forceinline__ u32x4 sv_pack(const float (&f)[8]) {
  return u32x4{sw_pack(f[0], f[1]), sw_pack(f[2], f[3]), sw_pack(f[4], f[5]), sw_pack(f[6], f[7])};
}
template <int CODEC>
__device__ __forceinline__ u32x2 sv_codes(const float (&f)[8], float s) {
  auto four = [&](int k) {
    if constexpr (CODEC == 0) return quant4<0>(f[k], f[k + 1], f[k + 2], f[k + 3], s);
    else return quant4_fnuz(f[k], f[k + 1], f[k + 2], f[k + 3], s);
  };
  return u32x2{four(0), four(4)};
}
__device__ __forceinline__ float sv_most(float m, const float (&f)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) m = fmaxf(m, fabsf(f[k]));
  return m;
}

// e^-|g|. -|g| log2(e) is taken as a rounded product t and the rest of it, which the product rule of the exponential puts
// back: within 2 ulp, in half the instructions of expf (the kernels are bound by their arithmetic: 46 instructions a value
// before). The hardware's exponential gives 0 below 2^-126; FAR (gates beyond 87) takes it 2^64 up there and
// rounds once on the way back, to fp32's spacing of 2^-149.
template <bool FAR>
__device__ __forceinline__ float sv_exp(float g) {
  const float x = FAR ? fmaxf(-fabsf(g), -104.0f) : -fabsf(g);   // below -104, e^x rounds to 0 in fp32
  const float t = x * 1.44269504f;
  const float rest = fmaf(x, 1.92596299e-8f, fmaf(x, 1.44269504f, -t));
  const bool low = FAR && t < -126.0f;
  float e = __builtin_amdgcn_exp2f(low ? t + 64.0f : t);   // exact: 64 brings t nearer to 0
  e = fmaf(e * rest, 0.693147182f, e);
  return low ? e * 0x1p-64f : e;
}

// sigmoid(g) and its complement sigmoid(-g) of eight gates, both with their own digits (1 - s keeps none where s nears 1).
// far: the lane may have a gate beyond 87; its whole wave then takes the exponentials again the longer way (16384 x 2048:
// forward 42 us so, as without the longer way; 44 with it for every value, 52 with a branch between the two).
__device__ __forceinline__ void sv_sigmoids(const float (&g)[8], bool far, float (&s)[8], float (&n)[8]) {
  float e[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) e[k] = sv_exp<false>(g[k]);
  if (__builtin_expect(__builtin_amdgcn_ballot_w64(far) != 0ull, 0)) {
#pragma unroll
    for (int k = 0; k < 8; ++k) e[k] = sv_exp<true>(g[k]);
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float rc = __builtin_amdgcn_rcpf(1.0f + e[k]), er = e[k] * rc;   // the denominator lies in [1, 2]
    const bool pos = g[k] >= 0.0f;
    s[k] = pos ? rc : er;
    n[k] = pos ? er : rc;
  }
}

// Keeps chunk c of a row's MX form; the four lanes of a block call it together.
__device__ __forceinline__ void sv_keep(const u32x4& v, int rule, uint8_t* q, uint8_t* s, int64_t c) {
  uint32_t m = pk_absmax_bf16(pk_absmax_bf16(0u, v.x), v.y);
  m = pk_fold(pk_absmax_bf16(pk_absmax_bf16(m, v.z), v.w));
  m = lane_max_xor<2, false>(lane_max_xor<1, false>(m));
  const int X = mx_exponent_bf16(m, rule);
  const float so = mx_scale_operand(X + 127);
  reinterpret_cast<u32x2*>(q)[c] = u32x2{mx_cvt4<true>(v.x, v.y, so), mx_cvt4<true>(v.z, v.w, so)};
  if ((threadIdx.x & 3) == 0) s[c >> 2] = (uint8_t)(X + 127);
}

// The eight values of a kept chunk.
__device__ __forceinline__ void sv_values(const u32x2& q, uint8_t e, float (&f)[8]) {
  const float so = mx_scale_operand(e);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t w = h ? q.y : q.x;
    const sv_f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w, so, false);
    const sv_f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w, so, true);
    f[4 * h] = a[0]; f[4 * h + 1] = a[1]; f[4 * h + 2] = b[0]; f[4 * h + 3] = b[1];
  }
}

__device__ __forceinline__ void sv_unpack(const u32x4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    f[2 * k] = bf16_lo(w[k]);
    f[2 * k + 1] = bf16_hi(w[k]);
  }
}

template <int CODEC, int TPR, int ITEMS>
__global__ __launch_bounds__(256) void swiglu_save_kernel(SaveArgs p) {
  constexpr int RPB = 256 / TPR;
  __shared__ float red[4];
  const int lt = threadIdx.x % TPR;
  const int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
  const bool valid = row < p.rows;
  const int64_t r = valid ? row : 0, F = p.F;
  const int nc = (int)(F >> 3);
  const u32x4* __restrict__ gr = reinterpret_cast<const u32x4*>(p.h1 + r * p.ld_h1);
  const u32x4* __restrict__ ur = reinterpret_cast<const u32x4*>(p.h1 + r * p.ld_h1 + F);
  uint8_t* const hq = p.hq + r * 2 * F;
  uint8_t* const hs = p.hs + r * (2 * F / 32);
  u32x2* const qr = reinterpret_cast<u32x2*>(p.q + r * F);
  u32x4* const ar = p.a2 != nullptr ? reinterpret_cast<u32x4*>(p.a2 + r * F) : nullptr;
  auto value = [&](const u32x4& g, const u32x4& u, float (&a)[8]) {
    float gf[8], uf[8];
    sv_unpack(g, gf);
    sv_unpack(u, uf);
    const uint32_t m = pk_fold(pk_absmax_bf16(pk_absmax_bf16(pk_absmax_bf16(pk_absmax_bf16(0u, g.x), g.y), g.z), g.w));
    float s[8], n[8];
    sv_sigmoids(gf, m > 0x42AEu, s, n);   // bf16(87)
#pragma unroll
    for (int k = 0; k < 8; ++k) a[k] = gf[k] * s[k] * uf[k];
  };
  auto first = [&](const u32x4& g, const u32x4& u, int c, float (&a)[8]) {
    sv_keep(g, p.rule, hq, hs, c);
    sv_keep(u, p.rule, hq + F, hs + F / 32, c);
    value(g, u, a);
    if (ar != nullptr) ar[c] = sv_pack(a);
  };
  float m = 0.0f;
  if constexpr (ITEMS > 0) {
    u32x4 gv[ITEMS], uv[ITEMS];
    float a[ITEMS][8];
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int c = i * TPR + lt;
      if (valid && c < nc) {
        gv[i] = gr[c];
        uv[i] = ur[c];
      }
    }
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int c = i * TPR + lt;
      if (valid && c < nc) {
        first(gv[i], uv[i], c, a[i]);
        m = sv_most(m, a[i]);
      }
    }
    const float s = scale_from_amax(sv_row_max<TPR>(m, red), CODEC);
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int c = i * TPR + lt;
      if (valid && c < nc) qr[c] = sv_codes<CODEC>(a[i], s);
    }
    if (valid && lt == 0) p.scale[row] = s;
  } else {
    float a[8];
    if (valid)
      for (int c = lt; c < nc; c += TPR) {
        first(gr[c], ur[c], c, a);
        m = sv_most(m, a);
      }
    const float s = scale_from_amax(sv_row_max<TPR>(m, red), CODEC);
    if (valid) {
      for (int c = lt; c < nc; c += TPR) {
        value(gr[c], ur[c], a);
        qr[c] = sv_codes<CODEC>(a, s);
      }
      if (lt == 0) p.scale[row] = s;
    }
  }
}

template <int CODEC, int TPR, int ITEMS>
__global__ __launch_bounds__(256) void swiglu_saved_bwd_kernel(SaveArgs p) {
  constexpr int RPB = 256 / TPR;
  __shared__ float red[4];
  const int lt = threadIdx.x % TPR;
  const int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
  const bool valid = row < p.rows;
  const int64_t r = valid ? row : 0, F = p.F;
  const int nc = (int)(F >> 3);
  const u32x4* __restrict__ dr = reinterpret_cast<const u32x4*>(p.da2 + r * F);
  const u32x2* __restrict__ gr = reinterpret_cast<const u32x2*>(p.hq + r * 2 * F);
  const u32x2* __restrict__ ur = reinterpret_cast<const u32x2*>(p.hq + r * 2 * F + F);
  const uint8_t* __restrict__ gs = p.hs + r * (2 * F / 32);
  const uint8_t* __restrict__ us = gs + F / 32;
  u32x4* const ar = p.a2 != nullptr ? reinterpret_cast<u32x4*>(p.a2 + r * F) : nullptr;
  u32x4* const og = p.dh1 != nullptr ? reinterpret_cast<u32x4*>(p.dh1 + r * 2 * F) : nullptr;
  u32x2* const qg = p.q != nullptr ? reinterpret_cast<u32x2*>(p.q + r * 2 * F) : nullptr;
  auto value = [&](const u32x4& d, const u32x2& g, const u32x2& u, int eg, int eu, float (&dg)[8], float (&du)[8],
                   float (&a)[8]) {
    float df[8], gf[8], uf[8];
    sv_unpack(d, df);
    sv_values(g, (uint8_t)eg, gf);
    sv_values(u, (uint8_t)eu, uf);
    float s[8], n[8];
    sv_sigmoids(gf, eg >= 125, s, n);   // 448 * 2^-3 is 56
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float gs_ = gf[k] * s[k];
      dg[k] = df[k] * uf[k] * s[k] * (1.0f + gf[k] * n[k]);
      du[k] = df[k] * gs_;
      a[k] = gs_ * uf[k];
    }
  };
  auto first = [&](const u32x4& d, const u32x2& g, const u32x2& u, int eg, int eu, int c, float (&dg)[8], float (&du)[8]) {
    float a[8];
    value(d, g, u, eg, eu, dg, du, a);
    if (og != nullptr) {
      og[c] = sv_pack(dg);
      og[nc + c] = sv_pack(du);
    }
    if (ar != nullptr) ar[c] = sv_pack(a);
  };
  float m = 0.0f;
  if constexpr (ITEMS > 0) {
    u32x4 dv[ITEMS];
    u32x2 gv[ITEMS], uv[ITEMS];
    int eg[ITEMS], eu[ITEMS];
    float dg[ITEMS][8], du[ITEMS][8];
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int c = i * TPR + lt;
      if (valid && c < nc) {
        dv[i] = dr[c];
        gv[i] = gr[c];
        uv[i] = ur[c];
        eg[i] = gs[c >> 2];
        eu[i] = us[c >> 2];
      }
    }
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int c = i * TPR + lt;
      if (valid && c < nc) {
        first(dv[i], gv[i], uv[i], eg[i], eu[i], c, dg[i], du[i]);
        m = sv_most(sv_most(m, dg[i]), du[i]);
      }
    }
    if (p.q == nullptr) return;   // uniform over the launch
    const float s = scale_from_amax(sv_row_max<TPR>(m, red), CODEC);
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int c = i * TPR + lt;
      if (valid && c < nc) {
        qg[c] = sv_codes<CODEC>(dg[i], s);
        qg[nc + c] = sv_codes<CODEC>(du[i], s);
      }
    }
    if (valid && lt == 0) p.scale[row] = s;
  } else {
    float dg[8], du[8], a[8];
    if (valid)
      for (int c = lt; c < nc; c += TPR) {
        first(dr[c], gr[c], ur[c], gs[c >> 2], us[c >> 2], c, dg, du);
        m = sv_most(sv_most(m, dg), du);
      }
    if (p.q == nullptr) return;
    const float s = scale_from_amax(sv_row_max<TPR>(m, red), CODEC);
    if (valid) {
      for (int c = lt; c < nc; c += TPR) {
        value(dr[c], gr[c], ur[c], gs[c >> 2], us[c >> 2], dg, du, a);
        qg[c] = sv_codes<CODEC>(dg, s);
        qg[nc + c] = sv_codes<CODEC>(du, s);
      }
      if (lt == 0) p.scale[row] = s;
    }
  }
}

template <bool BWD, int CODEC, int TPR, int ITEMS>
static hipError_t sv_launch(const SaveArgs& p, hipStream_t st) {
  const dim3 grid((unsigned)((p.rows + 256 / TPR - 1) / (256 / TPR)));
  if constexpr (BWD) hipLaunchKernelGGL((swiglu_saved_bwd_kernel<CODEC, TPR, ITEMS>), grid, dim3(256), 0, st, p);
  else hipLaunchKernelGGL((swiglu_save_kernel<CODEC, TPR, ITEMS>), grid, dim3(256), 0, st, p);
  return hipGetLastError();
}

template <bool BWD, int CODEC>
static hipError_t sv_pick(const SaveArgs& p, hipStream_t st) {
  const int64_t nc = p.F >> 3;
  // A whole workgroup a row of up to 256 chunks, one chunk a thread, where a wave's three or four chunks one after the other
  // take longer than idle threads cost: long rows (16384 x 2048: forward 53 -> 48 us, backward 76 -> 71), the backward
  // (49152 x 1408: 150 -> 143 us; 49152 x 800 88 -> 93 and not taken), few rows (509 x 1056: 5.0 -> 3.6 us). The forward
  // of 49152 x 1408 takes 93 us by waves, 109 by workgroups.
  if (nc <= 256 && (nc > 192 || (BWD && nc > 128) || (nc > 64 && p.rows < 2048))) return sv_launch<BWD, CODEC, 256, 1>(p, st);
  if (nc <= 16) return sv_launch<BWD, CODEC, 16, 1>(p, st);
  if (nc <= 32 && p.rows >= 2048) return sv_launch<BWD, CODEC, 16, 2>(p, st);   // 49152 x 256 27 -> 20 us; 500 rows 2.7 -> 3.3
  if (nc <= 64) return sv_launch<BWD, CODEC, 64, 1>(p, st);
  if (nc <= 128) return sv_launch<BWD, CODEC, 64, 2>(p, st);
  if constexpr (!BWD) {
    if (nc <= 192) return sv_launch<BWD, CODEC, 64, 3>(p, st);
  }
  if (nc <= 512) return sv_launch<BWD, CODEC, 256, 2>(p, st);
  if (nc <= 1024) return sv_launch<BWD, CODEC, 256, 4>(p, st);
  if (nc <= 2048) return sv_launch<BWD, CODEC, 256, 8>(p, st);
  return sv_launch<BWD, CODEC, 256, 0>(p, st);
}

hipError_t launch_swiglu_save(const uint16_t* h1, int64_t rows, int64_t F, int64_t ld_h1, int codec, int rule,
                              uint16_t* a2, uint8_t* q, float* scale, uint8_t* hq, uint8_t* hs, hipStream_t st) {
  if (rows == 0 || F == 0) return hipSuccess;
  const SaveArgs p{rows, F, ld_h1, h1, nullptr, hq, hs, rule, q, scale, a2, nullptr};
  return codec == 0 ? sv_pick<false, 0>(p, st) : sv_pick<false, 1>(p, st);
}

hipError_t launch_swiglu_saved_backward(const uint16_t* da2, const uint8_t* hq, const uint8_t* hs, int64_t rows, int64_t F,
                                        int codec, uint16_t* dh1, uint8_t* q, float* scale, uint16_t* a2, hipStream_t st) {
  if (rows == 0 || F == 0) return hipSuccess;
  const SaveArgs p{rows, F, 0, nullptr, da2, const_cast<uint8_t*>(hq), const_cast<uint8_t*>(hs), 0, q, scale, a2, dh1};
  return codec == 0 ? sv_pick<true, 0>(p, st) : sv_pick<true, 1>(p, st);
}

}  // namespace fp8moe
