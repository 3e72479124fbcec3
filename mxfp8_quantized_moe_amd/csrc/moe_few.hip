// The whole expert block of an MoE layer for a few tokens: gather, W1, SwiGLU,
// W2 and the weighted sum in two kernels, the weights in 8 bits and the
// activations in bf16.
//
//   [g | u] = x[t] W1[e]^T,  a[t, e] = bf16(silu(g) * u)          (first kernel)
//   y[t] = bf16(sum over the token's experts e of w[t, e] * a[t, e] W2[e]^T)   (second)
//
// Sums are fp32 on the matrix cores; a is rounded to bf16 because the matrix
// instruction takes it so (half a step, 2^-9 of its value on average, behind sums
// of thousands of products), y because the layer's stream is bf16.
//
// Every used expert's weights have to be read once, 3 K F bytes, and with a few tokens nothing else is of that
// size: the kernels stream weights.  A weight is the matrix instruction's row operand (16 rows of W a
// tile), the expert's tokens its 16 columns, so one read of a tile serves up to 64 tokens.  A lane loads 16 bytes of a
// row, 64 of a row lie in one instruction's four lane groups, and two v_mfma_f32_16x16x32_bf16
// take them: both operands permute the contraction alike, so no byte moves between lanes.  Codes become
// bf16 exactly (e4m3 and whole numbers up to 128 have at most eight significant bits); an e8m0 scale goes into
// that conversion, an fp32 scale divides the sum.  Activations come from L2 straight into registers.
//
// Tokens that choose one expert are found from the ids by every workgroup for itself: a bitmap of the
// experts in use, and for an expert a ballot over the tokens (at most 64, one a lane).  A
// token that names an expert twice is one column with the sum of its weights.
#include "device_common.hpp"
#include "kernels.hpp"
#include "swiglu_common.hpp"
#include "validate.hpp"

namespace fp8moe {

typedef __bf16 few_v8bf __attribute__((ext_vector_type(8)));
typedef __bf16 few_v2bf __attribute__((ext_vector_type(2)));
typedef float few_v4f __attribute__((ext_vector_type(4)));

enum { kFewFp8 = 0, kFewInt8 = 1, kFewMx = 2, kFewMxK4 = 3 };

struct FewParams {
  const uint16_t* x;      // [T][ld_x]
  int64_t ld_x;
  const int32_t* ids;     // [T][topk]
  const float* weights;   // [T][topk]
  const uint8_t* w1;      // [E][2F][K]
  const uint8_t* w2;      // [E][K][F]
  const void* s1;
  const void* s2;
  uint16_t* a2;           // [T * topk][F]: the row of a token's first slot of an expert
  uint16_t* y;            // [T][K]
  int T, topk, E, K, F;
};

// ---------------------------------------------------------------- who chose whom

struct FewIds {
  int n_act;                       // experts in use
  int ids[kFewMaxSlots];
  float w[kFewMaxSlots];
  uint32_t bits[32];               // experts in use, one bit each (E <= 1024)
  int act[kFewMaxSlots];           // the experts in use, in increasing order
};

// Fills `s` (every thread of the workgroup; ends with a barrier).
__device__ __forceinline__ void few_experts(const FewParams& p, FewIds& s) {
  const int t = threadIdx.x, S = p.T * p.topk;
  if (t < 32) s.bits[t] = 0;
  for (int i = t; i < S; i += blockDim.x) {
    s.ids[i] = p.ids[i];
    s.w[i] = p.weights[i];
  }
  __syncthreads();
  for (int i = t; i < S; i += blockDim.x) {
    const int e = s.ids[i];
    if (e >= 0 && e < p.E) atomicOr(&s.bits[e >> 5], 1u << (e & 31));
  }
  __syncthreads();
  if (t < 64) {
    uint32_t b = t < 32 ? s.bits[t] : 0u;
    int at = __popc(b);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up(at, d, 64);
      if (t >= d) at += o;
    }
    if (t == 31) s.n_act = at;
    for (at -= __popc(b); b != 0u; b &= b - 1u) s.act[at++] = 32 * t + __ffs(b) - 1;
  }
  __syncthreads();
}

struct FewList {
  int tok[64], slot[64];
  float w[64];
};

// LDS written by the wave's lanes so far is seen by its other lanes.
__device__ __forceinline__ void few_wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// The tokens of expert e, in order, by one wave; their count.
__device__ __forceinline__ int few_members(const FewParams& p, const FewIds& s, int e, FewList& l) {
  const int lane = threadIdx.x & 63;
  int first = -1;
  float w = 0.0f;
  if (lane < p.T) {
    for (int j = 0; j < p.topk; ++j) {
      const int i = lane * p.topk + j;
      if (s.ids[i] == e) {
        if (first < 0) first = i;
        w += s.w[i];
      }
    }
  }
  const unsigned long long m = __ballot(first >= 0);
  if (first >= 0) {
    const int at = __popcll(m & ((1ull << lane) - 1ull));
    l.tok[at] = lane;
    l.slot[at] = first;
    l.w[at] = w;
  }
  return __popcll(m);
}

// ---------------------------------------------------------------- products

// Sixteen bytes of a weight row and, for MX, the scale of their block.
__device__ __forceinline__ u32x4 few_load16(const uint8_t* q) {
  typedef unsigned int v4u __attribute__((ext_vector_type(4)));
  const v4u v = __builtin_nontemporal_load(reinterpret_cast<const v4u*>(q));
  return u32x4{v.x, v.y, v.z, v.w};
}

template <int FMT>
__device__ __forceinline__ few_v8bf few_bf16(uint32_t a, uint32_t b, float sc) {
  uint32_t o[4];
  if constexpr (FMT == kFewInt8) {
    const uint32_t w[2] = {a, b};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      // exact in bf16, so the upper halves of the fp32 patterns are the values
      const float f0 = (float)(signed char)(w[i] & 0xFFu), f1 = (float)(signed char)((w[i] >> 8) & 0xFFu);
      const float f2 = (float)(signed char)((w[i] >> 16) & 0xFFu), f3 = (float)(signed char)(w[i] >> 24);
      o[2 * i] = __builtin_amdgcn_perm(__float_as_uint(f1), __float_as_uint(f0), 0x07060302u);
      o[2 * i + 1] = __builtin_amdgcn_perm(__float_as_uint(f3), __float_as_uint(f2), 0x07060302u);
    }
  } else {
    o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, sc, false));
    o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, sc, true));
    o[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, sc, false));
    o[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, sc, true));
  }
  return __builtin_bit_cast(few_v8bf, u32x4{o[0], o[1], o[2], o[3]});
}

// A lane's row of an operand with MX scales: byte of block b at base + (b >> 2) * group + (b & 3) (K4), or base + b.
struct FewScale {
  const uint8_t* base;
  int64_t group;
};
template <int FMT>
__device__ __forceinline__ FewScale few_scale_row(const void* s, int64_t row, int64_t rows, int L) {
  const uint8_t* b = static_cast<const uint8_t*>(s);
  if constexpr (FMT == kFewMx) return FewScale{b + row * (L / 32), 0};
  else if constexpr (FMT == kFewMxK4) return FewScale{b + 4 * row, 4 * rows};
  else return FewScale{nullptr, 0};
}

// acc[r][b] += (tile r of 16 weight rows) x (16 tokens of block b) over the steps [s0, s1) of 64 contraction
// values; w and x are the lane's own rows.  Steps that pass L (a multiple of 16) load a valid chunk again and
// multiply it by zero.
template <int FMT, int R, int NB, int U>
__device__ __forceinline__ void few_dot(const uint8_t* const (&w)[R], const FewScale (&sc)[R],
                                        const uint16_t* const (&x)[NB], int L, int s0, int s1,
                                        few_v4f (&acc)[R][NB]) {
  const int kl = 16 * ((threadIdx.x & 63) >> 4);
  auto steps = [&](int s, auto whole_tag) {
    constexpr bool WHOLE = decltype(whole_tag)::value;
    u32x4 wv[U][R], xv[U][NB][2];
    float f[U][R];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int kk = 64 * (s + u) + kl;
      const int k = WHOLE ? kk : min(kk, L - 16);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        wv[u][r] = few_load16(w[r] + k);
        f[u][r] = 1.0f;
        if constexpr (FMT == kFewMx) f[u][r] = __uint_as_float((uint32_t)sc[r].base[k >> 5] << 23);
        if constexpr (FMT == kFewMxK4)
          f[u][r] = __uint_as_float((uint32_t)sc[r].base[(int64_t)(k >> 7) * sc[r].group + ((k >> 5) & 3)] << 23);
      }
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        xv[u][b][0] = *reinterpret_cast<const u32x4*>(x[b] + k);
        xv[u][b][1] = *reinterpret_cast<const u32x4*>(x[b] + k + 8);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if constexpr (!WHOLE) {
        const bool in = s + u < s1 && 64 * (s + u) + kl < L;
#pragma unroll
        for (int b = 0; b < NB; ++b)
          if (!in) xv[u][b][0] = xv[u][b][1] = u32x4{0, 0, 0, 0};
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const few_v8bf lo = few_bf16<FMT>(wv[u][r].x, wv[u][r].y, f[u][r]);
        const few_v8bf hi = few_bf16<FMT>(wv[u][r].z, wv[u][r].w, f[u][r]);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          acc[r][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(lo, __builtin_bit_cast(few_v8bf, xv[u][b][0]), acc[r][b], 0, 0, 0);
          acc[r][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(hi, __builtin_bit_cast(few_v8bf, xv[u][b][1]), acc[r][b], 0, 0, 0);
        }
      }
    }
  };
  int s = s0;
  for (; s + U <= s1 && 64 * (s + U) <= L; s += U) steps(s, std::true_type{});
  for (; s < s1; s += U) steps(s, std::false_type{});
}

// Calls f(NB) with the blocks of 16 that n tokens (1 .. 64) fill: 1, 2 or 4.
template <typename Fn>
__device__ __forceinline__ void few_blocks(int n, Fn&& f) {
  if (n <= 16) f(std::integral_constant<int, 1>{});
  else if (n <= 32) f(std::integral_constant<int, 2>{});
  else f(std::integral_constant<int, 4>{});
}

// ---------------------------------------------------------------- first kernel: a = silu(x Wg^T) * (x Wu^T)

// A workgroup takes 16 columns of F of one expert: 16 gate and 16 up rows of W1; its waves split K and
// add up through LDS.
template <int FMT, int W>
__global__ __launch_bounds__(64 * W) void few_up_kernel(FewParams p) {
  __shared__ FewIds ids;
  __shared__ FewList list;
  __shared__ int s_n;
  __shared__ few_v4f red[W][4][2][64];
  few_experts(p, ids);
  const int tiles = p.F / 16;
  const int rank = blockIdx.x / tiles, tile = blockIdx.x % tiles;
  if (rank >= ids.n_act) return;
  const int e = ids.act[rank];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if (wave == 0) {
    const int n = few_members(p, ids, e, list);
    if (lane == 0) s_n = n;
  }
  __syncthreads();
  const int n = s_n;
  const int64_t row = (int64_t)e * 2 * p.F + tile * 16 + (lane & 15);   // gate row; the up row lies F further
  const uint8_t* const w[2] = {p.w1 + row * p.K, p.w1 + (row + p.F) * p.K};
  const int64_t rows = (int64_t)p.E * 2 * p.F;
  const FewScale sc[2] = {few_scale_row<FMT>(p.s1, row, rows, p.K), few_scale_row<FMT>(p.s1, row + p.F, rows, p.K)};
  const int steps = (p.K + 63) / 64;
  const int s0 = steps * wave / W, s1 = steps * (wave + 1) / W;
  few_blocks(n, [&](auto nb_tag) {
    constexpr int NB = decltype(nb_tag)::value;
    const uint16_t* x[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) x[b] = p.x + (int64_t)list.tok[min(16 * b + (lane & 15), n - 1)] * p.ld_x;
    few_v4f acc[2][NB] = {};
    few_dot<FMT, 2, NB, NB == 4 ? 2 : 4>(w, sc, x, p.K, s0, s1, acc);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      red[wave][b][0][lane] = acc[0][b];
      red[wave][b][1][lane] = acc[1][b];
    }
  });
  __syncthreads();
  // lane l of a block: token l & 15, columns 4 (l >> 4) .. + 3 of the tile
  for (int i = threadIdx.x; i < ((n + 15) / 16) * 64; i += 64 * W) {
    const int b = i >> 6, l = i & 63, m = 16 * b + (l & 15);
    if (m >= n) continue;
    few_v4f g = red[0][b][0][l], u = red[0][b][1][l];
#pragma unroll
    for (int v = 1; v < W; ++v) {
      g += red[v][b][0][l];
      u += red[v][b][1][l];
    }
    const int c = tile * 16 + 4 * (l >> 4);
    float a[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float gj = g[j], uj = u[j];
      if constexpr (FMT == kFewFp8 || FMT == kFewInt8) {
        const float* s = static_cast<const float*>(p.s1) + (int64_t)e * 2 * p.F + c + j;
        gj = __fdiv_rn(gj, s[0]);
        uj = __fdiv_rn(uj, s[p.F]);
      }
      a[j] = gj * sw_sigmoid(gj) * uj;
    }
    *reinterpret_cast<u32x2*>(p.a2 + (int64_t)list.slot[m] * p.F + c) = u32x2{sw_pack(a[0], a[1]), sw_pack(a[2], a[3])};
  }
}

// ---------------------------------------------------------------- second kernel: y = sum of w * (a W2^T)

// A workgroup takes 16 columns of y: 16 rows of every used expert's W2.  The (expert, step) pairs of all experts in
// use form one sequence that its waves split evenly, each adding its products, times the router's weights, to its
// own sums in LDS; the waves' sums are added in order at the end, so no result depends on arrival.
template <int FMT, int W>
__global__ __launch_bounds__(64 * W) void few_down_kernel(FewParams p) {
  extern __shared__ __attribute__((aligned(16))) float few_y[];   // [W][T][16]
  __shared__ FewIds ids;
  __shared__ FewList lists[W];
  few_experts(p, ids);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  FewList& list = lists[wave];
  float* const mine = few_y + wave * p.T * 16;
  for (int i = lane; i < p.T * 16; i += 64) mine[i] = 0.0f;
  few_wave_sync();
  const int c0 = blockIdx.x * 16;
  const int per = (p.F + 63) / 64;   // steps of an expert
  const int total = ids.n_act * per;
  int at = (int)((int64_t)total * wave / W);
  const int end = (int)((int64_t)total * (wave + 1) / W);
  while (at < end) {
    const int rank = at / per, s0 = at - rank * per, s1 = min(per, s0 + end - at);
    const int e = __builtin_amdgcn_readfirstlane(ids.act[rank]);
    const int n = few_members(p, ids, e, list);
    few_wave_sync();
    const int64_t row = (int64_t)e * p.K + c0 + (lane & 15);
    const uint8_t* const w[1] = {p.w2 + row * p.F};
    const FewScale sc[1] = {few_scale_row<FMT>(p.s2, row, (int64_t)p.E * p.K, p.F)};
    few_v4f inv = {1.0f, 1.0f, 1.0f, 1.0f};
    if constexpr (FMT == kFewFp8 || FMT == kFewInt8) {
      const float* s = static_cast<const float*>(p.s2) + (int64_t)e * p.K + c0 + 4 * (lane >> 4);
#pragma unroll
      for (int j = 0; j < 4; ++j) inv[j] = s[j];
    }
    few_blocks(n, [&](auto nb_tag) {
      constexpr int NB = decltype(nb_tag)::value;
      const uint16_t* x[NB];
#pragma unroll
      for (int b = 0; b < NB; ++b) x[b] = p.a2 + (int64_t)list.slot[min(16 * b + (lane & 15), n - 1)] * p.F;
      few_v4f acc[1][NB] = {};
      few_dot<FMT, 1, NB, NB == 4 ? 2 : 4>(w, sc, x, p.F, s0, s1, acc);
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int m = 16 * b + (lane & 15);
        if (m >= n) continue;
        few_v4f* d = reinterpret_cast<few_v4f*>(mine + list.tok[m] * 16 + 4 * (lane >> 4));
        const float wt = list.w[m];
        few_v4f v = *d;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float o = acc[0][b][j];
          if constexpr (FMT == kFewFp8 || FMT == kFewInt8) o = __fdiv_rn(o, inv[j]);
          v[j] += wt * o;
        }
        *d = v;
      }
    });
    few_wave_sync();   // the list is rewritten for the next expert
    at += s1 - s0;
  }
  __syncthreads();
  // two columns a thread: four bytes of y
  for (int i = threadIdx.x; i < p.T * 8; i += 64 * W) {
    float a = 0.0f, b = 0.0f;
    for (int v = 0; v < W; ++v) {
      a += few_y[v * p.T * 16 + 2 * i];
      b += few_y[v * p.T * 16 + 2 * i + 1];
    }
    *reinterpret_cast<uint32_t*>(p.y + (int64_t)(i >> 3) * p.K + c0 + 2 * (i & 7)) = sw_pack(a, b);
  }
}

template <int FMT>
static hipError_t few_launch(const FewParams& p, hipStream_t st) {
  constexpr int W1 = 4, W2 = 8;
  const int64_t most = std::min<int64_t>(p.E, (int64_t)p.T * p.topk);
  if (p.F > 0) {
    hipLaunchKernelGGL((few_up_kernel<FMT, W1>), dim3((unsigned)(most * (p.F / 16))), dim3(64 * W1), 0, st, p);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  hipLaunchKernelGGL((few_down_kernel<FMT, W2>), dim3((unsigned)(p.K / 16)), dim3(64 * W2), W2 * p.T * 64, st, p);
  return hipGetLastError();
}

hipError_t launch_moe_few_tokens(const FewArgs& a, hipStream_t st) {
  if (a.tokens == 0 || a.K == 0) return hipSuccess;
  const FewParams p{a.x, a.ld_x, a.ids, a.weights, a.w1, a.w2, a.s1, a.s2, a.a2, a.y,
                    (int)a.tokens, a.topk, a.n_experts, (int)a.K, (int)a.F};
  switch (a.fmt) {
    case kFewFp8: return few_launch<kFewFp8>(p, st);
    case kFewInt8: return few_launch<kFewInt8>(p, st);
    case kFewMx: return few_launch<kFewMx>(p, st);
    default: return few_launch<kFewMxK4>(p, st);
  }
}

}  // namespace fp8moe
