// Products of 8-bit weight rows with the activations of a few tokens (at most 64), bound by the read of the weights.
//
// A weight is the matrix instruction's row operand (16 rows a tile), a token a column, so one read of a tile serves all
// tokens.  A lane loads 16 bytes of a row, and both operands permute the contraction alike.  With bf16 activations the codes become bf16 on the way (exactly: e4m3 and whole numbers up to 128 have at most
// eight significant bits) and two v_mfma_f32_16x16x32_bf16 take a lane's bytes; with whole-number activations
// one v_mfma_i32_16x16x64_i8 does.  Activations come from L2 straight into registers.
#pragma once

#include <type_traits>

#include "device_common.hpp"

namespace fp8moe {

typedef __bf16 few_v8bf __attribute__((ext_vector_type(8)));
typedef __bf16 few_v2bf __attribute__((ext_vector_type(2)));
typedef float few_v4f __attribute__((ext_vector_type(4)));

typedef int few_v4i __attribute__((ext_vector_type(4)));

// Weights: e4m3fn, whole numbers, e4m3fn with e8m0 scales (row-major, K4), all with bf16 activations; whole numbers
// with whole-number activations.
enum { kFewFp8 = 0, kFewInt8 = 1, kFewMx = 2, kFewMxK4 = 3, kFewInt8Both = 4 };

typedef float few_f4u __attribute__((ext_vector_type(4), aligned(4)));
typedef float few_v2f __attribute__((ext_vector_type(2)));

// Two fp32 values -> one word of two bf16 (round to nearest even).
__device__ __forceinline__ uint32_t few_pack(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(few_v2f{a, b}, few_v2bf));
}

// Sixteen bytes, streamed (non-temporal) or not.
template <bool STREAM>
__device__ __forceinline__ u32x4 few_load16(const uint8_t* base, uint32_t off) {
  typedef unsigned int v4u __attribute__((ext_vector_type(4)));
  if constexpr (STREAM) {
    const v4u v = __builtin_nontemporal_load(reinterpret_cast<const v4u*>(base + off));
    return u32x4{v.x, v.y, v.z, v.w};
  } else {
    return *reinterpret_cast<const u32x4*>(base + off);
  }
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

// A tile of weight rows and their e8m0 scales: first row, and the scale of its block b at
// (b >> 2) * group + (b & 3) (K4) or b.
struct FewTile {
  const uint8_t* w;
  const uint8_t* s;
  int64_t group;
};
template <int FMT>
__device__ __forceinline__ FewTile few_tile(const uint8_t* w, const void* s, int64_t row, int64_t rows, int L) {
  const uint8_t* b = static_cast<const uint8_t*>(s);
  if constexpr (FMT == kFewMx) return FewTile{w + row * L, b + row * (L / 32), 0};
  else if constexpr (FMT == kFewMxK4) return FewTile{w + row * L, b + 4 * row, 4 * rows};
  else return FewTile{w + row * L, nullptr, 0};
}

// Products of NT tiles of 16 weight rows with the tokens of an expert, over a wave's steps of 64 Q contraction values of
// rows of length L (a multiple of 16; a step that passes it loads a valid chunk again and multiplies it by zero).
//
// Q = 1: a tile is the instruction's 16 rows, NB blocks of 16 tokens its columns; a load takes 64 bytes of each
// row.  Q = 2, 4 (blocks of 16 / Q tokens): a tile is Q parts of 16 / Q rows, and an instruction takes each of a part's rows
// Q times, in neighbouring lanes with neighbouring chunks of 16 bytes, and each token's chunks in Q neighbouring
// columns.  Of the result only products of a row's q-th chunks with a token's q-th are of use; the sum over q, of
// neighbouring lanes, is the answer.  A load then takes 64 Q bytes of a row, whole cache lines, and the activations' loads
// are shared by the parts.
//
// The address unit takes four lanes a cycle where they lie in one line, and one or two where they do not, which is what bounds
// the loads of a CU: with a row's chunks 16 lanes apart 16 rows of 5120 x 5120 took 10.5 us, this way 8.2.  For Q = 1, where
// the instruction wants them 16 apart, neighbouring lanes load a row's four chunks and hand them over (400 rows of 4096 x
// 4096 34 -> 22 us; for Q = 2, pairs already, the handing over costs what it gains: 32 rows 8.6 -> 9.4).
//
// Part p has the rows p 4 / Q .. of each four, so that sums() leaves a lane four rows in order.
//
// W waves share the steps: ranges of them for Q > 1; for Q = 1 in turn, so that the other halves of the cache lines are
// asked for at the same time, by the next wave (509 rows in 11 groups of 1999 x 2064 20 -> 18 us; with whole lines
// 4 rows of 14336 x 4096 took 12.2 us in turn and 11.3 by ranges).
//
// STREAM: loads of whole cache lines are non-temporal, which leaves the activations in L2 (half lines that are streamed
// would be fetched twice).
template <int FMT, int NT, int NB, int Q, bool STREAM>
struct FewDot {
  static constexpr int ROWS = 16 / Q, PARTS = Q, R = NT * PARTS, STEP = 64 * Q, SUB = 4 / Q;
  using Acc = std::conditional_t<FMT == kFewInt8Both, few_v4i, few_v4f>;
  static constexpr int XB = FMT == kFewInt8Both ? 1 : 2;   // bytes of an activation
  // Steps whose loads are in flight together, by their registers (whole numbers 64 x 4096 x 4096: two 11.7 -> 10.4 us; bf16
  // 64 tokens, six of 16 experts 2048 x 1408: 62 -> 67).
  static constexpr int U = R * NB >= 16 ? 1 : R * NB >= 8 ? (XB == 1 && Q == 1 ? 2 : 1) : R * NB >= 4 ? 2 : 4;
  Acc acc[R][NB];

  // Of a block of rows or tokens, the one whose bytes the lane loads.
  static __device__ __forceinline__ int slot_of(int lane) { return Q == 1 ? lane >> 2 : (lane & 15) / Q; }

  // x: byte offset of the lane's row of activations from `xb`
  __device__ __forceinline__ void run(const FewTile (&tile)[NT], const void* xb, const uint32_t (&x)[NB], int L, int wave,
                                      int W) {
    const int all = (L + STEP - 1) / STEP, ds = Q == 1 ? W : 1;
    const int s0 = Q == 1 ? wave : all * wave / W, s1 = Q == 1 ? all : all * (wave + 1) / W;
    const int lane = threadIdx.x & 63;
    const uint32_t slot = slot_of(lane), row = Q == 1 ? slot : slot / SUB * 4 + slot % SUB, row_w = row * L;
    const int kl = Q == 1 ? 16 * (lane & 3) : 16 * Q * (lane >> 4) + 16 * (lane % Q);
    // the row and the chunk that the matrix instruction takes from the lane
    const uint32_t row_m = Q == 1 ? lane & 15 : row, row_s = FMT == kFewMxK4 ? 4 * row_m : row_m * (L / 32);
    const int kl_m = Q == 1 ? 16 * (lane >> 4) : kl, from = 16 * (lane & 15) + 4 * (lane >> 4);
    auto turn = [&](u32x4 v) {
      if constexpr (Q > 1) return v;
      return u32x4{(uint32_t)__builtin_amdgcn_ds_bpermute(from, v.x), (uint32_t)__builtin_amdgcn_ds_bpermute(from, v.y),
                   (uint32_t)__builtin_amdgcn_ds_bpermute(from, v.z), (uint32_t)__builtin_amdgcn_ds_bpermute(from, v.w)};
    };
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int b = 0; b < NB; ++b) acc[r][b] = Acc{0, 0, 0, 0};
    auto steps = [&](int s, auto whole_tag) {
      constexpr bool WHOLE = decltype(whole_tag)::value;
      u32x4 wv[U][R], xv[U][NB][XB];
      uint32_t e[U][R];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int kk = STEP * (s + u * ds) + kl;
        const uint32_t k = WHOLE ? kk : min(kk, L - 16), k_m = WHOLE ? kk - kl + kl_m : min(kk - kl + kl_m, L - 16);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const FewTile& t = tile[r / PARTS];
          wv[u][r] = few_load16<(STREAM && Q > 1)>(t.w + (int64_t)(r % PARTS) * SUB * L, row_w + k);
          if constexpr (FMT == kFewMx) e[u][r] = (t.s + (int64_t)(r % PARTS) * SUB * (L / 32))[row_s + (k_m >> 5)];
          if constexpr (FMT == kFewMxK4)
            e[u][r] = t.s[(int64_t)(k_m >> 7) * t.group + (row_s + (r % PARTS) * SUB * 4 + ((k_m >> 5) & 3))];
        }
#pragma unroll
        for (int b = 0; b < NB; ++b) {
#pragma unroll
          for (int h = 0; h < XB; ++h)
            xv[u][b][h] = few_load16<false>(static_cast<const uint8_t*>(xb), x[b] + XB * k + 16 * h);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if constexpr (!WHOLE) {
          const bool in = s + u * ds < s1 && STEP * (s + u * ds) + kl < L;
#pragma unroll
          for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int h = 0; h < XB; ++h)
              if (!in) xv[u][b][h] = u32x4{0, 0, 0, 0};
        }
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int h = 0; h < XB; ++h) xv[u][b][h] = turn(xv[u][b][h]);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          wv[u][r] = turn(wv[u][r]);
          if constexpr (FMT == kFewInt8Both) {
#pragma unroll
            for (int b = 0; b < NB; ++b)
              acc[r][b] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(few_v4i, wv[u][r]),
                                                                __builtin_bit_cast(few_v4i, xv[u][b][0]), acc[r][b], 0, 0, 0);
            continue;
          } else {
            float sc = 1.0f;
            if constexpr (FMT == kFewMx || FMT == kFewMxK4) sc = __uint_as_float(e[u][r] << 23);
            const few_v8bf lo = few_bf16<FMT>(wv[u][r].x, wv[u][r].y, sc);
            const few_v8bf hi = few_bf16<FMT>(wv[u][r].z, wv[u][r].w, sc);
#pragma unroll
            for (int b = 0; b < NB; ++b) {
              acc[r][b] =
                  __builtin_amdgcn_mfma_f32_16x16x32_bf16(lo, __builtin_bit_cast(few_v8bf, xv[u][b][0]), acc[r][b], 0, 0, 0);
              acc[r][b] =
                  __builtin_amdgcn_mfma_f32_16x16x32_bf16(hi, __builtin_bit_cast(few_v8bf, xv[u][b][1]), acc[r][b], 0, 0, 0);
            }
          }
        }
      }
    };
    int s = s0;
    for (; s + (U - 1) * ds < s1 && STEP * (s + (U - 1) * ds + 1) <= L; s += U * ds) steps(s, std::true_type{});
    for (; s < s1; s += U * ds) steps(s, std::false_type{});
  }

  // Rows 4 (lane >> 4) .. + 3 of tile h for token (lane & 15) / Q of block b, in all lanes.
  __device__ __forceinline__ Acc sums(int h, int b) const {
    if constexpr (Q == 1) return acc[h][b];
    const int q = threadIdx.x % Q;
    Acc t;
#pragma unroll
    for (int p = 0; p < PARTS; ++p) {
      const Acc& a = acc[h * PARTS + p][b];
      if constexpr (Q == 2) {
        t[2 * p] = pair_sum<0xB1>(q ? a[1] : a[0]);
        t[2 * p + 1] = pair_sum<0xB1>(q ? a[3] : a[2]);
      } else if constexpr (Q == 4) {
        t[p] = pair_sum<0x4E>(pair_sum<0xB1>(q & 2 ? (q & 1 ? a[3] : a[2]) : (q & 1 ? a[1] : a[0])));
      }
    }
    return t;
  }
  // v plus the value of the lane that the quad permutation names: 0xB1 the neighbour, 0x4E the next but one.
  template <int PERM, typename T>
  static __device__ __forceinline__ T pair_sum(T v) {
    return v + __builtin_bit_cast(T, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), PERM, 0xF, 0xF, true));
  }
};

// Calls f(NB, Q) for n tokens (1 .. 64) and NT tiles.  Whole lines (Q > 1) wherever their accumulators leave room for several
// waves: two tiles up to 32 tokens (32 rows of 4096 x 4096: 14.4 -> 8.7 us), four up to 16; beyond that they would be 128
// registers (64 rows in 64 groups, 2816 x 2048: 77 -> 128 us).
template <int NT, typename Fn>
__device__ __forceinline__ void few_blocks(int n, Fn&& f) {
  using I1 = std::integral_constant<int, 1>;
  using I2 = std::integral_constant<int, 2>;
  using I4 = std::integral_constant<int, 4>;
  if constexpr (NT == 2) {
    if (n <= 4) return f(I1{}, I4{});
  }
  if (n <= 8) f(I1{}, I2{});
  else if (n <= 16) f(I2{}, I2{});
  else if (n <= 32) f(std::integral_constant<int, NT == 2 ? 4 : 2>{}, std::integral_constant<int, NT == 2 ? 2 : 1>{});
  else f(I4{}, I1{});
}

}  // namespace fp8moe
