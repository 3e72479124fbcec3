// Root-mean-square norm of token rows with the residual's addition, quantized in
// the same pass (rowwise FP8 or MXFP8 1x32 blocks along the row), and its
// backward.
//
//   s = bf16(x + residual)            (s = x without a residual)
//   rstd = 1 / sqrt(sum(s^2) / C + eps)
//   f = (s * gamma) * rstd            fp32, never rounded before the cast
//   h = bf16(f);  codes of f under the rowwise or the MX recipe
//
// f is (s * gamma) * rstd in this order because rounding is monotonic: the
// largest |f| of a set is then exactly (largest |s * gamma|) * rstd, so the sum
// of squares and the maxima come out of one reduction, and no code depends on a
// second one.  The codes are cast from f itself, not from the bf16 copy h: one
// rounding instead of two.
//
// The row stays in registers from the load to the cast: TPR threads own one
// row, each with ITEMS 16-byte chunks of s.  HBM sees x and the residual once,
// and s, h and the codes once.
//
// Bound by HBM: with a residual, h and codes 9 bytes an element.  Measured on the
// GPU, medians (a 1 GiB device copy moves 5.2 TB/s): 16384 x 5120 with MX codes 141 us =
// 5.4 TB/s, 8192 x 4096 rowwise 52 us = 5.8 TB/s (part of its 302 MB stays in
// the last-level cache between passes).  16 rows of 7168: 3.9 us, latency.
#include "device_common.hpp"
#include "kernels.hpp"
#include "lane_groups.hpp"
#include "validate.hpp"

namespace fp8moe {

typedef float rn_f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 rn_bf16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(rn_f32x2{a, b}, rn_bf16x2));
}
__device__ __forceinline__ void unpack8(const u32x4& v, float (&f)[8]) {
  f[0] = bf16_lo(v.x); f[1] = bf16_hi(v.x);
  f[2] = bf16_lo(v.y); f[3] = bf16_hi(v.y);
  f[4] = bf16_lo(v.z); f[5] = bf16_hi(v.z);
  f[6] = bf16_lo(v.w); f[7] = bf16_hi(v.w);
}
__device__ __forceinline__ u32x4 pack8(const float (&f)[8]) {
  return u32x4{pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7])};
}

// Eight gamma values from column chunk c (GT 0: none, 1: fp32, 2: bf16).
template <int GT>
__device__ __forceinline__ void load_gamma(const void* __restrict__ gamma, int c, float (&g)[8]) {
  if constexpr (GT == 1) {
    const float4 a = reinterpret_cast<const float4*>(gamma)[2 * c], b = reinterpret_cast<const float4*>(gamma)[2 * c + 1];
    g[0] = a.x; g[1] = a.y; g[2] = a.z; g[3] = a.w;
    g[4] = b.x; g[5] = b.y; g[6] = b.z; g[7] = b.w;
  } else if constexpr (GT == 2) {
    unpack8(reinterpret_cast<const u32x4*>(gamma)[c], g);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) g[k] = 1.0f;
  }
}

struct NormFwd {
  const uint16_t* x;
  const uint16_t* res;    // or null
  const void* gamma;      // or null
  int64_t rows, ld_x, ld_r;
  int64_t row0;           // first row of this launch
  int nchunk;             // cols / 8
  float inv_c, eps;
  uint16_t* sum;          // [rows][cols], written with a residual
  uint16_t* h;            // [rows][cols] or null
  uint8_t* q;             // [rows][cols] or null
  float* scale;           // rowwise scales [rows]
  uint8_t* sc;            // MX scales
  float* rstd;            // [rows] or null
  int layout;             // MX scale layout
};

// Four e4m3fnuz codes of f * s.  A code's value is half the e4m3fn value of the same code, so enc_fnuz(y) =
// enc_fn(2y) up to 224 (doubling is exact); 2y above the tie 464 is 240 (0x7F: the low bit on top of the clamped
// 448's 0x7E), and a zero result drops its sign.  On whole words: 24 operations for four codes, where four single
// codes take over 40.
__device__ __forceinline__ uint32_t quant4_fnuz(float a, float b, float c, float d, float s) {
  const float s2 = 2.0f * s;
  const float y[4] = {a * s2, b * s2, c * s2, d * s2};
  float k[4];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    k[i] = __builtin_amdgcn_fmed3f(y[i], -448.0f, 448.0f);
    top |= fabsf(y[i]) > 464.0f ? 1u << (8 * i) : 0u;
  }
  const uint32_t w = cvt_fn_pair<true>(k[2], k[3], cvt_fn_pair<false>(k[0], k[1], 0u)) | top;
  const uint32_t mag = w & 0x7F7F7F7Fu;
  return mag | (w & (mag + 0x7F7F7F7Fu) & 0x80808080u);   // the sign where the magnitude is not 0
}

// FMT 0: rowwise e4m3fn, 1: rowwise e4m3fnuz, 2: MX floor rule, 3: MX ceil rule, 4: no codes.
template <int TPR, int ITEMS, int FMT, int GT>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void rmsnorm_kernel(NormFwd p) {
  constexpr int NT = TPR > 256 ? TPR : 256, RPB = NT / TPR, WAVES = TPR / 64;
  constexpr bool MX = FMT == 2 || FMT == 3, ROWWISE = FMT < 2;
  __shared__ float red_s[TPR > 64 ? WAVES : 1];
  __shared__ uint32_t red_m[TPR > 64 ? WAVES : 1];
  const int lt = threadIdx.x % TPR;
  const int64_t row = p.row0 + (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
  const bool valid = row < p.rows;
  const int64_t r = valid ? row : 0;
  const int64_t cols = (int64_t)p.nchunk * 8;
  const u32x4* xr = reinterpret_cast<const u32x4*>(p.x + r * p.ld_x);   // the sum may be written over it
  u32x4 v[ITEMS];
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int c = i * TPR + lt;
    v[i] = valid && c < p.nchunk ? xr[c] : u32x4{0, 0, 0, 0};
  }
  if (p.res != nullptr) {
    const u32x4* rr = reinterpret_cast<const u32x4*>(p.res + r * p.ld_r);
    u32x4* so = reinterpret_cast<u32x4*>(p.sum + r * cols);   // may be x's rows or the residual's
    u32x4 w[ITEMS];
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int c = i * TPR + lt;
      w[i] = valid && c < p.nchunk ? rr[c] : u32x4{0, 0, 0, 0};
    }
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int c = i * TPR + lt;
      float a[8], b[8];
      unpack8(v[i], a);
      unpack8(w[i], b);
#pragma unroll
      for (int k = 0; k < 8; ++k) a[k] += b[k];
      v[i] = pack8(a);
      if (valid && c < p.nchunk) so[c] = v[i];
    }
  }
  float ss = 0.0f;
  float f[ITEMS][8];   // s * gamma
  float am[ITEMS];     // its largest magnitude in each chunk
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int c = i * TPR + lt;
    float g[8];
    unpack8(v[i], f[i]);
    am[i] = 0.0f;
    if (c < p.nchunk) {
      load_gamma<GT>(p.gamma, c, g);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        ss += f[i][k] * f[i][k];
        f[i][k] *= g[k];
        am[i] = fmaxf(am[i], fabsf(f[i][k]));
      }
    }
  }
  uint32_t mb = 0;   // the row's largest magnitude (non-negative: its bits are ordered like the values)
  if constexpr (ROWWISE) {
    float rm = 0.0f;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) rm = fmaxf(rm, am[i]);
    mb = __float_as_uint(rm);
  }
  if constexpr (TPR <= 64) {
    ss = group_sum_f32<TPR>(ss);
    if constexpr (ROWWISE) mb = group_max_u32<TPR>(mb);
  } else {
    ss = group_sum_f32<64>(ss);
    if constexpr (ROWWISE) mb = group_max_u32<64>(mb);
    const int w = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
      red_s[w] = ss;
      red_m[w] = mb;
    }
    __syncthreads();
    float part[WAVES];
#pragma unroll
    for (int i = 0; i < WAVES; ++i) part[i] = red_s[i];
#pragma unroll
    for (int n = WAVES / 2; n >= 1; n /= 2)
#pragma unroll
      for (int i = 0; i < n; ++i) part[i] += part[i + n];
    ss = part[0];
    if constexpr (ROWWISE) {
#pragma unroll
      for (int i = 0; i < WAVES; ++i) mb = max(mb, red_m[i]);
    }
  }
  const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(ss * p.inv_c + p.eps));
  float scale = 0.0f;
  if constexpr (ROWWISE) scale = scale_from_amax(__uint_as_float(mb) * rstd, FMT);
  if (valid && lt == 0) {
    if (p.rstd != nullptr) p.rstd[row] = rstd;
    if constexpr (ROWWISE) p.scale[row] = scale;
  }
  const int nb = p.nchunk >> 2;   // 32-blocks per row (MX)
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int c = i * TPR + lt;
    const bool in = valid && c < p.nchunk;
    float(&a)[8] = f[i];
#pragma unroll
    for (int k = 0; k < 8; ++k) a[k] *= rstd;
    if (in && p.h != nullptr) reinterpret_cast<u32x4*>(p.h + r * cols)[c] = pack8(a);
    if constexpr (ROWWISE) {
      auto four = [&](int k) {
        if constexpr (FMT == 0) return quant4<0>(a[k], a[k + 1], a[k + 2], a[k + 3], scale);
        else return quant4_fnuz(a[k], a[k + 1], a[k + 2], a[k + 3], scale);
      };
      if (in) reinterpret_cast<u32x2*>(p.q + r * cols)[c] = u32x2{four(0), four(4)};
    }
    if constexpr (MX) {
      // four lanes hold one block (chunks 4b .. 4b+3; TPR is a multiple of four)
      const uint32_t bm = lane_max_xor<2, false>(lane_max_xor<1, false>(__float_as_uint(am[i] * rstd)));
      const int X = mx_exponent(bm, FMT - 2);
      const float inv = exp2_neg(X);
      if (in)
        reinterpret_cast<u32x2*>(p.q + r * cols)[c] =
            u32x2{quant4<0>(a[0], a[1], a[2], a[3], inv), quant4<0>(a[4], a[5], a[6], a[7], inv)};
      if (in && (lt & 3) == 0) {
        const int b = c >> 2;
        const uint8_t code = (uint8_t)(X + 127);
        if (p.layout == 0) {
          p.sc[r * nb + b] = code;
        } else {
          uint8_t* const word = p.sc + ((int64_t)(b >> 2) * p.rows + r) * 4;
          word[b & 3] = code;
          if (b == nb - 1)
            for (int t = (b & 3) + 1; t < 4; ++t) word[t] = 0;
        }
      }
    }
  }
}

// Rows of one launch: 2^23 workgroups of 256 threads stay within the 32 bits of a grid's thread count.
constexpr int64_t kNormLaunchRows = 1 << 23;

template <int TPR, int ITEMS, int FMT>
static hipError_t launch_fwd_g(const NormFwd& p, int gt, hipStream_t st) {
  constexpr int NT = TPR > 256 ? TPR : 256, RPB = NT / TPR;
  const int64_t rows = p.rows - p.row0 < kNormLaunchRows ? p.rows - p.row0 : kNormLaunchRows;
  const dim3 grid((unsigned)((rows + RPB - 1) / RPB)), block(NT);
  if (gt == 0) hipLaunchKernelGGL((rmsnorm_kernel<TPR, ITEMS, FMT, 0>), grid, block, 0, st, p);
  else if (gt == 1) hipLaunchKernelGGL((rmsnorm_kernel<TPR, ITEMS, FMT, 1>), grid, block, 0, st, p);
  else hipLaunchKernelGGL((rmsnorm_kernel<TPR, ITEMS, FMT, 2>), grid, block, 0, st, p);
  return hipGetLastError();
}

template <int FMT>
static hipError_t launch_fwd(const NormFwd& p, int gt, hipStream_t st) {
  const int n = p.nchunk;   // <= 2048
  if (n <= 16) return launch_fwd_g<16, 1, FMT>(p, gt, st);
  if (n <= 32) return launch_fwd_g<16, 2, FMT>(p, gt, st);
  if (n <= 64) return launch_fwd_g<16, 4, FMT>(p, gt, st);
  if (n <= 128) return launch_fwd_g<64, 2, FMT>(p, gt, st);
  if (n <= 256) return launch_fwd_g<64, 4, FMT>(p, gt, st);
  // Few long rows (at most two workgroups a compute unit): a row's latency counts (16 x 7168: 3.7 us, with 256
  // threads a row 5.0 us; beyond, 256 threads keep more rows in flight).
  if (p.rows <= 512) {
    if (n <= 1024) return launch_fwd_g<1024, 1, FMT>(p, gt, st);
    return launch_fwd_g<1024, 2, FMT>(p, gt, st);
  }
  // A second chunk of 256 threads would be mostly empty (4093 x 2056, codes only: 9.4 us, so 10.5 us).
  if (n <= 320) return launch_fwd_g<64, 5, FMT>(p, gt, st);
  if (n <= 512) return launch_fwd_g<256, 2, FMT>(p, gt, st);
  if (n <= 768) return launch_fwd_g<256, 3, FMT>(p, gt, st);
  if (n <= 1024) return launch_fwd_g<256, 4, FMT>(p, gt, st);
  return launch_fwd_g<256, 8, FMT>(p, gt, st);
}

static_assert(kNormMaxCols == 256 * 8 * 8, "256 threads hold eight chunks of eight columns each");

hipError_t launch_rmsnorm_quantize(const NormArgs& a, hipStream_t st) {
  if (a.rows == 0) return hipSuccess;
  NormFwd p;
  p.x = a.x;
  p.res = a.res;
  p.gamma = a.gamma;
  p.rows = a.rows;
  p.ld_x = a.ld_x;
  p.ld_r = a.ld_r;
  p.nchunk = (int)(a.cols >> 3);
  p.inv_c = 1.0f / (float)a.cols;
  p.eps = a.eps;
  p.sum = a.sum;
  p.h = a.h;
  p.q = a.q;
  p.scale = a.scale;
  p.sc = a.sc;
  p.rstd = a.rstd;
  p.layout = a.layout;
  const int gt = a.gamma == nullptr ? 0 : (a.gamma_bf16 ? 2 : 1);
  for (p.row0 = 0; p.row0 < a.rows; p.row0 += kNormLaunchRows) {
    hipError_t e;
    switch (a.fmt) {
      case 0: e = launch_fwd<0>(p, gt, st); break;
      case 1: e = launch_fwd<1>(p, gt, st); break;
      case 2: e = launch_fwd<2>(p, gt, st); break;
      case 3: e = launch_fwd<3>(p, gt, st); break;
      default: e = launch_fwd<4>(p, gt, st); break;
    }
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// ---------------------------------------------------------------- backward
//
// With n = s * rstd and g = dh * gamma:
//   dx = rstd * (g - n * mean(g * n)) (+ dsum),   dgamma = sum over rows of dh * n.
// A workgroup walks rows with a stride of the grid and keeps its columns' share of
// dgamma in registers (fp32); the shares go to the workspace, one row per
// workgroup, and a second kernel adds them in a fixed order.  Bound by HBM: 8 bytes
// an element with dsum.  512 workgroups: 16384 x 5120 takes 137-143 us (medians of five
// traces; 4.8 TB/s) + 5 us for the shares; 1024 take 132 + 14 where 512 took 135 + 5, and
// where only 768 fit (8192 x 7168) 119 instead of 97.  Loading dsum with the other rows
// instead of after the row's sum, and three chunks a thread instead of four, brought both
// kernels together from 195 us to about 145.

struct NormBwd {
  const uint16_t* dh;
  const uint16_t* s;
  const float* rstd;
  const void* gamma;
  const uint16_t* dsum;   // or null
  int64_t rows;
  int nchunk;
  float inv_c;
  uint16_t* dx;
  float* part;            // [grid][cols] or null (no dgamma wanted)
};

template <int TPR, int ITEMS, int GT>
__global__ __launch_bounds__(256) void rmsnorm_bwd_kernel(NormBwd p) {
  constexpr int RPB = 256 / TPR;
  __shared__ float red[2][4];
  const int lt = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  const int64_t cols = (int64_t)p.nchunk * 8;
  float acc[ITEMS][8];
#pragma unroll
  for (int i = 0; i < ITEMS; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[i][k] = 0.0f;
  int turn = 0;
  for (int64_t base = (int64_t)blockIdx.x * RPB; base < p.rows; base += (int64_t)gridDim.x * RPB, turn ^= 1) {
    const int64_t row = base + sub;
    const bool valid = row < p.rows;
    const int64_t r = valid ? row : 0;
    const float rstd = valid ? p.rstd[r] : 0.0f;
    u32x4 dv[ITEMS], sv[ITEMS], ev[ITEMS];
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int c = i * TPR + lt;
      const bool in = valid && c < p.nchunk;
      dv[i] = in ? reinterpret_cast<const u32x4*>(p.dh + r * cols)[c] : u32x4{0, 0, 0, 0};
      sv[i] = in ? reinterpret_cast<const u32x4*>(p.s + r * cols)[c] : u32x4{0, 0, 0, 0};
      ev[i] = u32x4{0, 0, 0, 0};
    }
    if (p.dsum != nullptr) {
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) {
        const int c = i * TPR + lt;
        if (valid && c < p.nchunk) ev[i] = reinterpret_cast<const u32x4*>(p.dsum + r * cols)[c];
      }
    }
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int c = i * TPR + lt;
      float d[8], n[8], g[8];
      unpack8(dv[i], d);
      unpack8(sv[i], n);
      if (c < p.nchunk) {
        load_gamma<GT>(p.gamma, c, g);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float nk = n[k] * rstd;
          acc[i][k] += d[k] * nk;
          dot += d[k] * g[k] * nk;
        }
      }
    }
    if constexpr (TPR <= 64) {
      dot = group_sum_f32<TPR>(dot);
    } else {
      dot = group_sum_f32<64>(dot);
      // two sets of slots in turn: the next row's write cannot meet this row's reads
      if ((threadIdx.x & 63) == 0) red[turn][threadIdx.x >> 6] = dot;
      __syncthreads();
      dot = (red[turn][0] + red[turn][1]) + (red[turn][2] + red[turn][3]);
    }
    const float m = dot * p.inv_c;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int c = i * TPR + lt;
      if (valid && c < p.nchunk) {
        float d[8], n[8], g[8], e[8];
        unpack8(dv[i], d);
        unpack8(sv[i], n);
        load_gamma<GT>(p.gamma, c, g);
        unpack8(ev[i], e);
#pragma unroll
        for (int k = 0; k < 8; ++k) e[k] += rstd * (d[k] * g[k] - n[k] * rstd * m);
        reinterpret_cast<u32x4*>(p.dx + r * cols)[c] = pack8(e);
      }
    }
  }
  if (p.part == nullptr) return;   // uniform
  float* const out = p.part + (int64_t)blockIdx.x * cols;
  if constexpr (RPB == 1) {
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int c = i * TPR + lt;
      if (c < p.nchunk) {
        reinterpret_cast<float4*>(out)[2 * c] = float4{acc[i][0], acc[i][1], acc[i][2], acc[i][3]};
        reinterpret_cast<float4*>(out)[2 * c + 1] = float4{acc[i][4], acc[i][5], acc[i][6], acc[i][7]};
      }
    }
  } else {
    // the RPB row slots of a column add up through LDS, one chunk set at a time
    __shared__ float sh[256 * 8];
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      __syncthreads();
#pragma unroll
      for (int k = 0; k < 8; ++k) sh[(sub * TPR + lt) * 8 + k] = acc[i][k];
      __syncthreads();
      for (int e = threadIdx.x; e < TPR * 8; e += 256) {
        float t = 0.0f;
#pragma unroll
        for (int u = 0; u < RPB; ++u) t += sh[u * TPR * 8 + e];
        const int64_t col = (int64_t)i * TPR * 8 + e;
        if (col < cols) out[col] = t;
      }
    }
  }
}

// dgamma[c] = the workgroups' shares added in a fixed order: 64 columns a workgroup, whose 16 waves each add every
// 16th share, eight loads in flight.
__global__ __launch_bounds__(1024) void rmsnorm_dgamma_kernel(const float* __restrict__ part, int n, int64_t cols,
                                                              float* __restrict__ dgamma) {
  constexpr int B = 8;
  __shared__ float sh[16][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * 64 + lane;
  float t = 0.0f;
  if (c < cols) {
    for (int i0 = w; i0 < n; i0 += 16 * B) {
      float v[B];
      // a share past the last one loads the last one again: no branch between the loads
#pragma unroll
      for (int i = 0; i < B; ++i) v[i] = part[(int64_t)min(i0 + 16 * i, n - 1) * cols + c];
#pragma unroll
      for (int i = 0; i < B; ++i) t += i0 + 16 * i < n ? v[i] : 0.0f;
    }
  }
  sh[w][lane] = t;
  __syncthreads();
  if (w == 0 && c < cols) {
    t = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) t += sh[i][lane];
    dgamma[c] = t;
  }
}

template <int TPR, int ITEMS>
static hipError_t launch_bwd_g(const NormBwd& p, int gt, int grid, hipStream_t st) {
  if (gt == 0) hipLaunchKernelGGL((rmsnorm_bwd_kernel<TPR, ITEMS, 0>), dim3(grid), dim3(256), 0, st, p);
  else if (gt == 1) hipLaunchKernelGGL((rmsnorm_bwd_kernel<TPR, ITEMS, 1>), dim3(grid), dim3(256), 0, st, p);
  else hipLaunchKernelGGL((rmsnorm_bwd_kernel<TPR, ITEMS, 2>), dim3(grid), dim3(256), 0, st, p);
  return hipGetLastError();
}

hipError_t launch_rmsnorm_backward(const uint16_t* dh, const uint16_t* s, const float* rstd, const void* gamma,
                                   bool gamma_bf16, const uint16_t* dsum, int64_t rows, int64_t cols, uint16_t* dx,
                                   float* dgamma, float* workspace, hipStream_t st) {
  if (rows == 0 && dgamma == nullptr) return hipSuccess;
  NormBwd p;
  p.dh = dh;
  p.s = s;
  p.rstd = rstd;
  p.gamma = gamma;
  p.dsum = dsum;
  p.rows = rows;
  p.nchunk = (int)(cols >> 3);
  p.inv_c = 1.0f / (float)cols;
  p.dx = dx;
  p.part = dgamma != nullptr ? workspace : nullptr;
  const int gt = gamma == nullptr ? 0 : (gamma_bf16 ? 2 : 1);
  const int grid = norm_bwd_blocks(rows, cols);
  auto pick = [&](auto tpr_tag) -> hipError_t {
    constexpr int TPR = decltype(tpr_tag)::value;
    const int items = (p.nchunk + TPR - 1) / TPR;
    if (items <= 1) return launch_bwd_g<TPR, 1>(p, gt, grid, st);
    if (items <= 2) return launch_bwd_g<TPR, 2>(p, gt, grid, st);
    if (items <= 3) return launch_bwd_g<TPR, 3>(p, gt, grid, st);
    if constexpr (TPR == 256)
      if (items > 4) return launch_bwd_g<TPR, 8>(p, gt, grid, st);
    return launch_bwd_g<TPR, 4>(p, gt, grid, st);
  };
  hipError_t e = hipSuccess;
  if (grid > 0) {
    if (p.nchunk <= 64) e = pick(std::integral_constant<int, 16>{});
    else if (p.nchunk <= 256) e = pick(std::integral_constant<int, 64>{});
    else e = pick(std::integral_constant<int, 256>{});
  }
  if (e != hipSuccess || dgamma == nullptr) return e;
  hipLaunchKernelGGL(rmsnorm_dgamma_kernel, dim3((unsigned)((cols + 63) / 64)), dim3(1024), 0, st, workspace, grid,
                     cols, dgamma);
  return hipGetLastError();
}

}  // namespace fp8moe
