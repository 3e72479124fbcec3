// Router gate in front of moe_route, the load-balance loss over its choices, and
// their backward.
//
//   score = softmax(logits) or sigmoid(logits) of a token's eligible experts
//   ids   = the topk experts of largest key (the logit, or score + bias), in
//           decreasing order, equal keys to the lower index
//   w     = route_scale * score (divided by the chosen scores' sum)
//   loss  = coef / S * sum over sequences s and experts i of f_si * P_si, with
//           f = count * E / (topk * n), P the mean of the scores normalised to sum 1
//
// A logit that is NaN or -inf makes its expert ineligible for the token; +inf
// counts as the largest finite value.
//
// Layout: LPT lanes (4, 16 or 64) share a token, so a wave takes up to 16 tokens.
// Lane l of the group holds VPL logits: where rows are aligned (VEC), in chunks of
// four, experts 4 (l + LPT c) + 0..3, which are 16-byte loads and stores; else
// experts l + LPT v, so that the lanes of each 4-byte access are neighbours.  Sums
// and maxima over a token then take 2, 4 or 6 VALU lane steps, shared by the wave's
// tokens.
//
// Selection, first round: a key is an fp32 value (the logit, or score + bias) made
// sortable as an unsigned integer, its low four bits replaced by the complement of
// the value's place in the lane.  Each lane sorts its VPL keys once (a network of
// max/min pairs); a choice is then the group's maximum of the list heads, equal
// heads go to the lower place and then to the lower lane, which is the lower
// expert, and the lane that owned the head moves its list up.  The chosen experts'
// exact values are formed anyway, for the weights: where two consecutive choices
// are in the wrong order or, with a bias, closer than the rounding of fp32 keys
// allows, or where the first key left out may be as large as the last choice, the
// wave selects again in a second round over whole keys: the exact logit, or
// score + bias formed in 64 bits, equal keys to the lower expert.
//
// Measured on the GPU, fp32 logits, medians (copy rate 5.2 TB/s).  Choice, 65536 x 256 top
// 8: 21 us without a bias, 25 us with one and sigmoid scores, 26-29 us with softmax scores
// (71 MB: 14 us); bound by the vector ALU's issue, busy 87% of the time (661 vector
// operations a wave of four tokens: about 260 for scores and keys, 126 for the sorting
// network, 17 a choice).  A wave a token took 120 us, looking for close choices once
// instead of after each choice 71 -> 47 us, the place in the key 47 -> 41 us, a second
// round that takes a token at a time 41 -> 31 us.  With the loss 29 us (softmax) + 10 us
// for its sums; 8192 x 64 top 6: 6.5 + 6 us.  Backward, 65536 x 256 (140 MB: 27 us): 28 us
// softmax, bound by HBM, 32 us sigmoid (vector ALU 65% busy); 8192 x 64: 5.8 us.
//
// Where the second round takes every token the choice costs four times as much, and more:
// constant logits 80 us (65536 x 256 top 8, no bias), a softmax row held by one expert under a bias
// of zeros 108 us (the tolerance of close keys is absolute).
#include "device_common.hpp"
#include "kernels.hpp"
#include "lane_groups.hpp"
#include "validate.hpp"

namespace fp8moe {

static_assert(kGateMaxExperts == 1024, "64 lanes hold 16 logits each");

constexpr float kFltMax = 3.402823466e38f;
typedef float gt_f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 gt_bf16x2 __attribute__((ext_vector_type(2)));

// Orders the wave's own LDS accesses for the compiler (the hardware keeps them in order).
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// ---------------------------------------------------------------- logits

// NaN as -inf (the maximum of a NaN and a number is the number), at most the largest finite value.
__device__ __forceinline__ float gate_clean(float v) { return fminf(fmaxf(v, -INFINITY), kFltMax); }

template <bool BF16>
__device__ __forceinline__ float gate_logit(const void* __restrict__ logits, int64_t at) {
  if constexpr (BF16) return gate_clean(__uint_as_float((uint32_t)static_cast<const uint16_t*>(logits)[at] << 16));
  else return gate_clean(static_cast<const float*>(logits)[at]);
}

// The expert of the lane's value v.
template <int LPT, bool VEC>
__device__ __forceinline__ int expert_at(int l, int v) {
  return VEC ? 4 * (l + LPT * (v >> 2)) + (v & 3) : l + LPT * v;
}

// The lane's VPL logits of a row starting at element `row` (-inf past E or when off).  VEC: E and the row
// stride are multiples of four and every array of experts starts aligned, so a chunk is one load.  RAW: not cleaned.
template <int LPT, int VPL, bool BF16, bool VEC, bool RAW = false>
__device__ __forceinline__ void gate_load(const void* __restrict__ logits, int64_t row, int E, int l, bool on,
                                          float (&z)[VPL]) {
  if constexpr (VEC) {
#pragma unroll
    for (int c = 0; c < VPL / 4; ++c) {
      const int e0 = 4 * (l + LPT * c);
      float4 w = float4{-INFINITY, -INFINITY, -INFINITY, -INFINITY};
      if (on && e0 < E) {
        if constexpr (BF16) {
          const u32x2 h = *reinterpret_cast<const u32x2*>(static_cast<const uint16_t*>(logits) + row + e0);
          w = float4{bf16_lo(h.x), bf16_hi(h.x), bf16_lo(h.y), bf16_hi(h.y)};
        } else {
          w = *reinterpret_cast<const float4*>(static_cast<const float*>(logits) + row + e0);
        }
      }
      z[4 * c] = w.x; z[4 * c + 1] = w.y; z[4 * c + 2] = w.z; z[4 * c + 3] = w.w;
    }
  } else {
    const int n = on ? E : 0;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      const int e = expert_at<LPT, VEC>(l, v);
      z[v] = -INFINITY;
      if (e < n) {
        if constexpr (BF16) z[v] = __uint_as_float((uint32_t)static_cast<const uint16_t*>(logits)[row + e] << 16);
        else z[v] = static_cast<const float*>(logits)[row + e];
      }
    }
  }
  // All loads have left before the first is cleaned (the compiler would clean each in its own branch, one wait a load).
#pragma unroll
  for (int v = 0; v < VPL; ++v) asm volatile("" : "+v"(z[v]));
  if constexpr (!RAW) {
#pragma unroll
    for (int v = 0; v < VPL; ++v) z[v] = gate_clean(z[v]);
  }
}

// fp32 vector of the experts (a bias, the loss's derivative), 0 past E.
template <int LPT, int VPL, bool VEC>
__device__ __forceinline__ void gate_load_vec(const float* __restrict__ x, int E, int l, float (&out)[VPL]) {
  if constexpr (VEC) {
#pragma unroll
    for (int c = 0; c < VPL / 4; ++c) {
      const int e0 = 4 * (l + LPT * c);
      const float4 w = e0 < E ? *reinterpret_cast<const float4*>(x + e0) : float4{0.f, 0.f, 0.f, 0.f};
      out[4 * c] = w.x; out[4 * c + 1] = w.y; out[4 * c + 2] = w.z; out[4 * c + 3] = w.w;
    }
  } else {
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      const int e = expert_at<LPT, VEC>(l, v);
      out[v] = e < E ? x[e] : 0.0f;
    }
  }
}

__device__ __forceinline__ float sigmoid_f32(float z) { return __builtin_amdgcn_rcpf(1.0f + __expf(-z)); }

// A sigmoid score s, its complement 1 - s = sigmoid(-z) and its derivative s (1 - s), each to a few roundings of itself (1 - s
// formed from a rounded s has no digits left from a logit of 17 on).
struct Sigmoid {
  float s, comp, slope;
};
__device__ __forceinline__ Sigmoid sigmoid_parts(float z) {
  const float e = __expf(-fabsf(z));   // 0 for infinities
  const float big = __builtin_amdgcn_rcpf(1.0f + e), small = e * big;
  return z >= 0.0f ? Sigmoid{big, small, small * big} : Sigmoid{small, big, small * big};
}

// A score on the scale of the largest of its kind: without the factor exp(c), c the largest logit (a sigmoid's at most 0).
// The largest is at least a half, so their sum cannot vanish and their ratios hold where every score is below the fp32
// range: chosen experts' where a bias chooses 100 below the others, a sigmoid row's from logits of -87 on.
template <bool SIGMOID>
__device__ __forceinline__ float scaled_score(float z, float c) {
  if constexpr (SIGMOID) return __expf(fminf(z, 0.0f) - c) * __builtin_amdgcn_rcpf(1.0f + __expf(-fabsf(z)));
  else return __expf(z - c);
}
// Renormalised weights are taken on that scale where the chosen scores' sum is below this.  With a larger sum, a score that
// falls below the fp32 range is below 2^-102 of it.
constexpr float kLowChosen = 0x1p-24f;

// Scores of the lane's logits, the softmax's before its division: m is the row's maximum, total their sum
// over the token.
template <int LPT, int VPL, bool SIGMOID>
__device__ __forceinline__ void gate_scores(const float (&z)[VPL], float (&s)[VPL], float& m, float& total) {
  m = -kFltMax;
  if constexpr (!SIGMOID) {
#pragma unroll
    for (int v = 0; v < VPL; ++v) m = fmaxf(m, z[v]);
    m = group_max_f32<LPT>(m);
  }
  total = 0.0f;
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    s[v] = SIGMOID ? sigmoid_f32(z[v]) : __expf(z[v] - m);   // 0 for -inf
    total += s[v];
  }
  total = group_sum_f32<LPT>(total);
}

// A sigmoid token's scores and one over their sum where the sum is below kLowTotal, on the scale of the row's largest logit
// (all are negative).  With a sum of kLowTotal and more a score below the fp32 range is below 2^-125 of it.  A row whose
// sigmoids are 0 in 64 bits (all logits below kLeastSigmoid, as those of a row masked by the type's lowest value are) has no
// share of the loss.
constexpr float kLowTotal = 0.5f;
constexpr float kLeastSigmoid = -709.78f;
// The path is rare: it reads the logits again, one at a time, and passes the scores through the token's LDS row `mine`
// (W floats), so that the kernels around it keep their registers.
template <int LPT, int VPL, bool BF16, bool VEC>
__device__ __forceinline__ void low_sigmoid_scores(const void* __restrict__ logits, int64_t row, int E, int l, bool low,
                                                   float* mine, float (&s)[VPL], float& inv) {
  const int n = low ? E : 0;
  float m = -kFltMax, total = 0.0f;
#pragma unroll 1
  for (int v = 0; v < VPL; ++v) {
    const int e = expert_at<LPT, VEC>(l, v);
    if (e < n) m = fmaxf(m, gate_logit<BF16>(logits, row + e));
  }
  m = group_max_f32<LPT>(m);
#pragma unroll 1
  for (int v = 0; v < VPL; ++v) {
    const int e = expert_at<LPT, VEC>(l, v);
    const float z = e < n ? gate_logit<BF16>(logits, row + e) : -INFINITY;
    const float w = scaled_score<true>(z, m);   // 0 for -inf
    mine[e] = w;
    total += w;
  }
  total = group_sum_f32<LPT>(total);
  wave_lds_fence();
  if (low) {
    inv = total > 0.0f && m >= kLeastSigmoid ? __fdiv_rn(1.0f, total) : 0.0f;
#pragma unroll
    for (int v = 0; v < VPL; ++v) s[v] = mine[expert_at<LPT, VEC>(l, v)];
  }
  wave_lds_fence();
}

// ---------------------------------------------------------------- keys

// A value that is not -0.
__device__ __forceinline__ uint32_t sortable_nz(float v) {
  const uint32_t b = __float_as_uint(v);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ uint32_t sortable(float v) { return sortable_nz(v + 0.0f); }   // -0 -> +0
__device__ __forceinline__ float sorted_value(uint32_t s) {
  return __uint_as_float(s ^ ((int32_t)s < 0 ? 0x80000000u : 0xFFFFFFFFu));
}
constexpr uint32_t kLeast32 = 0x00800000u;   // -FLT_MAX; -inf (no eligible expert) and 0 (an emptied list) are below

// Descending order by Batcher's odd-even merge network.
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return max(a, b); }
__device__ __forceinline__ uint32_t smaller(uint32_t a, uint32_t b) { return min(a, b); }
template <typename T, int N>
__device__ __forceinline__ void sort_desc(T (&k)[N]) {
#pragma unroll
  for (int p = 1; p < N; p *= 2)
#pragma unroll
    for (int q = p; q >= 1; q /= 2)
#pragma unroll
      for (int j = q % p; j + q < N; j += 2 * q)
#pragma unroll
        for (int i = 0; i < q; ++i)
          if (i + j + q < N && (i + j) / (2 * p) == (i + j + q) / (2 * p)) {
            const T a = k[i + j], b = k[i + j + q];
            k[i + j] = larger(a, b);
            k[i + j + q] = smaller(a, b);
          }
}

// Whether this is the lowest lane of its group of LPT for which `is` holds; it holds somewhere in every group, and all
// lanes are here.  On the wave's mask, by scalar operations: one taken from each group's bits clears its lowest set
// one and, as no group is empty, borrows nothing from the next group.
template <int LPT>
__device__ __forceinline__ bool lowest_lane(bool is) {
  constexpr uint64_t kOnes = LPT == 64 ? 1u : LPT == 16 ? 0x0001000100010001u : 0x1111111111111111u;
  const uint64_t all = __ballot(is);
  return __builtin_amdgcn_inverse_ballot_w64(all & ~(all - kOnes));
}

// The list without its head where `take`: of a sorted list only the first KEEP keys are needed.
template <int KEEP, typename T, int N>
__device__ __forceinline__ void move_up(T (&k)[N], bool take) {
#pragma unroll
  for (int v = 0; v < KEEP - 1; ++v) {
    const T here = k[v], next = k[v + 1];
    k[v] = take ? next : here;
  }
  const T here = k[KEEP - 1];
  k[KEEP - 1] = take ? T(0) : here;
}

// f(KEEP) with the keys a lane can lose to topk choices (the loop over the choices is picked once, not each step of it).
template <int N, typename F>
__device__ __forceinline__ void with_keep(int topk, F&& f) {
  if constexpr (N > 8) {
    if (topk <= 8) {
      f(std::integral_constant<int, 8>{});
      return;
    }
  }
  f(std::integral_constant<int, N>{});
}

// The second round for one token (row, wave-uniform), by a whole wave: its choices go to slot[0 .. topk).
// m: the row's largest logit (softmax).  A key is the logit, or score + bias in 64 bits, all of them: the wave takes the
// largest and then the lowest expert that holds it, an exchange of its own (an index in the key's low bits would make
// keys equal that are 2^-41 of their value apart).
template <int VPL, bool BF16, bool SIGMOID, bool VEC>
__device__ __forceinline__ void select_exact(const void* __restrict__ logits, int64_t row, int E,
                                             const float* __restrict__ bias, float m, int topk, int* slot) {
  const int lane = threadIdx.x & 63, first = expert_at<64, VEC>(lane, 0);   // the lane's experts lie at the same distances
  float z[VPL];
  double key[VPL];   // -inf: not eligible, or chosen before
  gate_load<64, VPL, BF16, VEC>(logits, row, E, lane, true, z);
  if (bias == nullptr) {
#pragma unroll
    for (int v = 0; v < VPL; ++v) key[v] = (double)z[v];
  } else {
    float b[VPL];
    gate_load_vec<64, VPL, VEC>(bias, E, lane, b);
    double total = 0.0;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      key[v] = SIGMOID ? 1.0 / (1.0 + exp(-(double)z[v])) : exp((double)z[v] - (double)m);
      total += key[v];
    }
    if constexpr (!SIGMOID) total = group_sum_f64<64>(total);
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      const double k = (SIGMOID ? key[v] : key[v] / total) + (double)b[v];
      key[v] = z[v] > -INFINITY && b[v] > -INFINITY ? k : -(double)INFINITY;   // a NaN of the bias is not above -inf
    }
  }
  for (int j = 0; j < topk; ++j) {
    double best = key[0];
#pragma unroll
    for (int v = 1; v < VPL; ++v) best = fmax(best, key[v]);
    best = group_max_f64<64>(best);
    int at = kGateMaxExperts - first;   // the lane's lowest expert that holds it, from its first; none: past the last there is
#pragma unroll
    for (int v = VPL - 1; v >= 0; --v) at = key[v] == best ? expert_at<64, VEC>(0, v) : at;
    const int id = kGateMaxExperts - (int)group_most_u32<64>((uint32_t)(kGateMaxExperts - first - at));
    if (lane == 0) slot[j] = best > -(double)INFINITY ? id : -1;
#pragma unroll
    for (int v = 0; v < VPL; ++v) key[v] = expert_at<64, VEC>(0, v) == id - first ? -(double)INFINITY : key[v];
  }
}

// ---------------------------------------------------------------- work units
//
// A workgroup takes one unit: up to `chunk` tokens of one sequence (or of the
// tokens behind the last one).

struct TokenRange {
  int seq;      // -1: behind the last sequence (or past the end)
  int t0, t1;
};
__device__ __forceinline__ TokenRange gate_unit(const int32_t* __restrict__ offs, int S, int T, int u, int chunk) {
  auto chunks = [chunk](int lo, int hi) { return gate_chunks(lo, hi, chunk); };
  auto len = [](int lo, int hi) { return hi - lo; };
  const Unit un = find_unit_quant<256>(offs, S, T, u, chunks, len);
  if (un.e >= 0) {
    const int t0 = un.lo + un.j * chunk;
    return TokenRange{un.e, t0, gate_chunk_end(t0, un.hi, chunk)};
  }
  const int64_t t0 = un.pbase + (int64_t)un.j * chunk;   // pbase: the end of the last sequence
  return t0 < T ? TokenRange{-1, (int)t0, (int)min(t0 + chunk, (int64_t)T)} : TokenRange{-1, 0, 0};
}

// ---------------------------------------------------------------- forward

struct GateFwd {
  const void* logits;
  int64_t ld;
  int T, E, topk, renorm, chunk, S;
  const float* bias;
  const uint8_t* mask;
  float route_scale;
  int32_t* ids;            // written by the gate, read by the loss alone
  float* weights;
  const int32_t* offs;
  float* part_p;           // [units][E] sums of normalised scores
  int32_t* part_c;         // [units][E] slots choosing the expert
  int32_t* part_n;         // [units] tokens that count
  uint64_t* total;         // the loss kernel's sum and counter, cleared here
};

template <int LPT, int VPL, bool BF16, bool VEC, bool SIGMOID, bool GATE, bool BAL>
__global__ __launch_bounds__(256) void gate_kernel(GateFwd p) {
  constexpr int TPW = 64 / LPT;                  // tokens a wave takes at a time
  constexpr int W = LPT * VPL;
  // Places that different lanes' experts of equal value are ordered by, before the lane: all of them, or (a lane's four
  // in a chunk come before the next lane's) the chunks.
  constexpr uint32_t kCompare = VEC ? ~3u : ~0u;
  constexpr int SLOTS = W < kGateMaxTopk ? W : kGateMaxTopk;
  // A token's choices: lane and place, then the expert; its logit's bits, then its score's.  (A wave's rows hold at least
  // 64 of each.)
  __shared__ int s_slot[GATE ? 256 / LPT * SLOTS : 1];
  __shared__ int s_val[GATE ? 256 / LPT * SLOTS : 1];
  __shared__ int s_cnt[BAL ? W : 1];
  __shared__ __attribute__((aligned(16))) float s_sum[BAL ? 256 * VPL : 1];
  __shared__ int s_n[4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l = lane % LPT, g = lane / LPT;
  TokenRange rg;
  if constexpr (BAL) {
    rg = gate_unit(p.offs, p.S, p.T, blockIdx.x, p.chunk);
    if (blockIdx.x == 0 && threadIdx.x < 2) p.total[threadIdx.x] = 0;
    for (int e = threadIdx.x; e < p.E; e += 256) s_cnt[e] = 0;
    __syncthreads();
  } else {
    const int64_t t0 = (int64_t)blockIdx.x * p.chunk;
    rg = TokenRange{0, (int)t0, (int)min(t0 + p.chunk, (int64_t)p.T)};
  }
  const bool counted = BAL && rg.seq >= 0;   // workgroup-uniform
  float acc[VPL];
  int n = 0;
#pragma unroll
  for (int v = 0; v < VPL; ++v) acc[v] = 0.0f;

  for (int base = rg.t0 + wave * TPW; base < rg.t1; base += 4 * TPW) {   // wave-uniform
    const int t = base + g;
    const bool live = t < rg.t1;
    const bool on = live && (p.mask == nullptr || p.mask[t] != 0);
    const int64_t row = (int64_t)t * p.ld, slot0 = (int64_t)t * p.topk;
    float z[VPL], s[VPL], m, total;
    // Sigmoid keys with a bias take the logits as they are, a sixth fewer operations a logit.
    constexpr bool RAW = SIGMOID && GATE && !BAL;
    gate_load<LPT, VPL, BF16, VEC, RAW>(p.logits, row, p.E, l, on, z);
    gate_scores<LPT, VPL, SIGMOID>(z, s, m, total);
    const float inv = total > 0.0f ? __fdiv_rn(1.0f, total) : 0.0f;

    if constexpr (GATE) {
      const bool biased = p.bias != nullptr;
      int* const slot = s_slot + (wave * TPW + g) * SLOTS;
      int* const val = s_val + (wave * TPW + g) * SLOTS;
      bool close = false;
      {
        uint32_t key[VPL];
        if (!biased) {
#pragma unroll
          for (int v = 0; v < VPL; ++v) key[v] = (sortable(RAW ? gate_clean(z[v]) : z[v]) & ~15u) | (uint32_t)(15 - v);
        } else {
          float b[VPL];
          gate_load_vec<LPT, VPL, VEC>(p.bias, p.E, l, b);
#pragma unroll
          for (int v = 0; v < VPL; ++v) {
            // NaN (of the bias) is below all; +inf stays, the checks below see it as close to the largest finite
            // value; a sum of a score, which is not -0, is not -0
            const float k = fmaxf((SIGMOID ? s[v] : s[v] * inv) + b[v], -INFINITY);
            key[v] = (sortable_nz(z[v] > -INFINITY ? k : -INFINITY) & ~15u) | (uint32_t)(15 - v);
          }
        }
        sort_desc(key);
        const uint32_t ninth = key[VPL > 8 ? 8 : 0];
        // The lane that owns a choice writes it; the others write beside it (a place of their own among the wave's
        // values, which are not in use yet): without a branch the lists move by selects.
        int* const aside = s_val + wave * TPW * SLOTS + lane;
        with_keep<VPL>(p.topk, [&](auto keep) {
          for (int j = 0; j < p.topk; ++j) {
            const uint32_t head = key[0] & kCompare;
            const uint32_t best = group_most_u32<LPT>(head);
            const bool mine = lowest_lane<LPT>(head == best);
            *(mine ? slot + j : aside) = best >= kLeast32 ? (int)((key[0] & 15u) | (uint32_t)(l << 4)) : -1;
            move_up<decltype(keep)::value>(key, mine);
          }
        });
        const uint32_t left = group_most_u32<LPT>(key[0] & kCompare);
        // with_keep keeps eight of a lane's keys for topk 8: one that gave all eight away and had a ninth cannot
        // tell what is left
        if constexpr (VPL > 8) close = p.topk == 8 && key[0] == 0u && ninth >= kLeast32;
        wave_lds_fence();
        // Error of an fp32 key with a bias, u = 2^-24: a sigmoid is within 5 u (its exponential's relative error
        // |z| 3 u + 2 u enters times s (1 - s) <= min(1/4, e^-|z|)), a softmax score within 55 u (exponent
        // e^-x (3 x + 2) u, the sum's error up to 50 u), the sum with the bias rounds by u |key|.  Two keys can
        // swap below twice that.  A key without its low four bits is lower by less than 2^-19 of its value.
        const float tol = SIGMOID ? 0x1p-20f : 0x1p-17f;
        float before = 0.0f;   // slot j0 - 1
        int before_id = -1;
        for (int j0 = 0; j0 < p.topk; j0 += LPT) {
          const int j = j0 + l;
          const int raw = j < p.topk ? slot[j] : -1;
          const int id = raw >= 0 ? expert_at<LPT, VEC>(raw >> 4, 15 - (raw & 15)) : -1;
          float x = -INFINITY;
          if (id >= 0) {
            x = gate_logit<BF16>(p.logits, row + id);
            slot[j] = id;
            val[j] = __float_as_int(x);
            if (biased) x = gate_clean((SIGMOID ? sigmoid_f32(x) : __expf(x - m) * inv) + p.bias[id]);
          }
          const float xp = __shfl_up(x, 1, LPT);
          const int ip = __shfl_up(id, 1, LPT);
          const float xb = l > 0 ? xp : before;
          const int ib = l > 0 ? ip : before_id;
          if (ib >= 0 && id >= 0)
            close = close || (biased ? xb - x <= tol * (1.0f + fabsf(x)) : !(xb > x || (xb == x && ib < id)));
          if (j == p.topk - 1 && left >= kLeast32) {
            const float y = sorted_value(left & ~15u);
            close = close || (biased ? x - y <= tol * (1.0f + fabsf(y)) + 0x1p-18f * fabsf(y)
                                     : !BF16 && ((sortable(x) ^ left) & ~15u) == 0);
          }
          before = __shfl(x, LPT - 1, LPT);
          before_id = __shfl(id, LPT - 1, LPT);
        }
      }
      // Second round: the whole wave takes one token after another of those that need it, so its wide keys
      // occupy few registers beside the first round's.
      for (uint64_t todo = __ballot(close); todo != 0;) {
        const int gc = (__ffsll((unsigned long long)todo) - 1) / LPT;   // wave-uniform
        todo &= ~(LPT == 64 ? ~0ull : ((1ull << (LPT & 63)) - 1) << (gc * (LPT & 63)));
        select_exact<W <= 256 ? 4 : VPL, BF16, SIGMOID, VEC>(p.logits, (int64_t)(base + gc) * p.ld, p.E, p.bias,
                                                             __shfl(m, gc * LPT, 64), p.topk,
                                                             s_slot + (wave * TPW + gc) * SLOTS);
        wave_lds_fence();
        if (g == gc)
          for (int j = l; j < p.topk; j += LPT)
            if (slot[j] >= 0) val[j] = __float_as_int(gate_logit<BF16>(p.logits, row + slot[j]));
      }
      wave_lds_fence();
      float ws = 0.0f, c = -INFINITY;   // c: the lane's largest chosen logit, where a score of it is small
      for (int j = l; j < p.topk; j += LPT) {
        const float zj = __int_as_float(val[j]);
        const float w = slot[j] < 0 ? 0.0f : SIGMOID ? sigmoid_f32(zj) : __expf(zj - m);
        c = slot[j] < 0 ? c : fmaxf(c, zj);
        val[j] = __float_as_int(w);
        ws += w;
      }
      if (p.renorm) {
        ws = group_sum_f32<LPT>(ws);
        if (__ballot(ws < kLowChosen && c > -INFINITY) != 0) {   // wave-uniform, rare
          c = group_max_f32<LPT>(c);
          if constexpr (SIGMOID) c = fminf(c, 0.0f);
          float scaled = 0.0f;
          if (ws < kLowChosen) {
            for (int j = l; j < p.topk; j += LPT) {
              const float w = slot[j] < 0 ? 0.0f : scaled_score<SIGMOID>(gate_logit<BF16>(p.logits, row + slot[j]), c);
              val[j] = __float_as_int(w);
              scaled += w;
            }
          }
          scaled = group_sum_f32<LPT>(scaled);
          ws = ws < kLowChosen ? scaled : ws;
        }
      }
      for (int j = l; j < p.topk; j += LPT) {
        float w = __int_as_float(val[j]);
        if (p.renorm) w = ws > 0.0f ? __fdiv_rn(w, ws) : 0.0f;   // exactly 1 for a single choice
        else if constexpr (!SIGMOID) w *= inv;
        if (live) {
          p.ids[slot0 + j] = slot[j];
          p.weights[slot0 + j] = w * p.route_scale;
        }
      }
    }
    if constexpr (BAL) {
      if (counted && on) {
        for (int j = l; j < p.topk; j += LPT) {
          int id;
          if constexpr (GATE) id = s_slot[(wave * TPW + g) * SLOTS + j];
          else id = p.ids[slot0 + j];
          if (id >= 0 && id < p.E) atomicAdd(&s_cnt[id], 1);
        }
        if (l == 0) ++n;
      }
      float share = inv;
      if constexpr (SIGMOID) {
        const bool low = on && total < kLowTotal;
        if (counted && __ballot(low) != 0)   // wave-uniform
          low_sigmoid_scores<LPT, VPL, BF16, VEC>(p.logits, row, p.E, l, low, s_sum + (wave * TPW + g) * W, s, share);
      }
      if (counted && on) {
#pragma unroll
        for (int v = 0; v < VPL; ++v) acc[v] += s[v] * share;
      }
    }
    if constexpr (GATE) wave_lds_fence();   // before the next token's choices
  }
  if constexpr (BAL) {
    constexpr int NG = 256 / LPT;   // token groups of the workgroup, each with its share of the sums
#pragma unroll
    for (int v = 0; v < VPL; ++v) s_sum[(wave * TPW + g) * W + expert_at<LPT, VEC>(l, v)] = acc[v];
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) n += __shfl_xor(n, o, 64);
    if (lane == 0) s_n[wave] = n;
    __syncthreads();
    if (!counted) return;
    const int64_t at = (int64_t)blockIdx.x * p.E;
    for (int e = threadIdx.x; e < p.E; e += 256) {
      float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < NG; ++i) sum[i & 3] += s_sum[i * W + e];
      p.part_p[at + e] = (sum[0] + sum[1]) + (sum[2] + sum[3]);
      p.part_c[at + e] = s_cnt[e];
    }
    if (threadIdx.x == 0) p.part_n[blockIdx.x] = (s_n[0] + s_n[1]) + (s_n[2] + s_n[3]);
  }
}

// ---------------------------------------------------------------- the loss from the units' sums

constexpr int kLossSlice = 32;   // experts a workgroup of the loss kernel adds up

struct GateLoss {
  int T, E, topk, chunk, S;
  float coef;
  const int32_t* offs;
  const float* part_p;
  const int32_t* part_c;
  const int32_t* part_n;
  uint64_t* total;     // sum over slices in units of 2^-53, slices that added theirs; 0 on entry
  float* loss;
  int32_t* counts;     // [S][E]
  float* dprob;        // [S][E]
};

// First unit and unit count of sequence s (workgroup-wide; the rule of find_unit).
template <int NT>
__device__ __forceinline__ void seq_units(const int32_t* __restrict__ offs, int S, int T, int s, int chunk, int& first,
                                          int& count) {
  if (offs == nullptr) {
    first = 0;
    count = gate_chunks(0, T, chunk);
    return;
  }
  if (S <= 64) {   // every wave on its own, no barrier
    const int lane = threadIdx.x & 63;
    int hi = lane < S ? clamp_off(offs[lane], T) : 0;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(hi, d, 64);
      if (lane >= d) hi = max(hi, o);
    }
    int lo = __shfl_up(hi, 1, 64);
    if (lane == 0) lo = 0;
    const int cnt = lane < S ? gate_chunks(lo, hi, chunk) : 0;
    int incl = cnt;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(incl, d, 64);
      if (lane >= d) incl += o;
    }
    first = __shfl(incl - cnt, s, 64);
    count = __shfl(cnt, s, 64);
    return;
  }
  __shared__ int tmp[NT / 64], s_hi[NT], s_total, s_first, s_count;
  const int t = threadIdx.x;
  int base = 0, carry = 0;
  for (int g0 = 0; g0 <= s; g0 += NT) {
    const int e = g0 + t;
    const int v = e < S ? clamp_off(offs[e], T) : 0;
    const int hi = max(block_scan_max<NT>(v, tmp), carry);
    s_hi[t] = hi;
    __syncthreads();
    const int lo = t == 0 ? carry : s_hi[t - 1];
    const int cnt = e < S ? gate_chunks(lo, hi, chunk) : 0;
    const int incl = block_scan_sum<NT>(cnt, tmp) + base;
    if (e == s) {
      s_first = incl - cnt;
      s_count = cnt;
    }
    if (t == NT - 1) s_total = incl;
    __syncthreads();
    base = s_total;
    carry = s_hi[NT - 1];
    __syncthreads();
  }
  first = s_first;
  count = s_count;
}

// One workgroup for 32 experts of a sequence: its 32 half-waves each add every 32nd
// unit, eight loads in flight, in 64 bits.  The sum over slices and sequences of
// f P / S, at most E <= 2^10, is kept as a whole number of 2^-53 (the at most 2^21
// terms' roundings are 2^-33 together): additions of whole numbers do not depend on their order.
// Each addition has come back before its slice counts as arrived, so the last one finds them all.
__global__ __launch_bounds__(1024) void gate_loss_kernel(GateLoss p) {
  constexpr int B = 8;
  __shared__ double sh_p[32][kLossSlice];
  __shared__ int sh_c[32][kLossSlice], sh_n[16];
  const int s = blockIdx.y, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int i0 = threadIdx.x / kLossSlice, ie = threadIdx.x % kLossSlice;
  const int e = blockIdx.x * kLossSlice + ie;
  int first, count;
  seq_units<1024>(p.offs, p.S, p.T, s, p.chunk, first, count);
  int n = 0;
  for (int u = threadIdx.x; u < count; u += 1024) n += p.part_n[first + u];
  double sum = 0.0;
  int c = 0;
  if (e < p.E) {
    for (int u0 = i0; u0 < count; u0 += 32 * B) {
      float q[B];
      int d[B];
#pragma unroll
      for (int i = 0; i < B; ++i) {
        // a unit past the last one loads the last one again: no branch between the loads
        const int64_t at = (int64_t)(first + min(u0 + 32 * i, count - 1)) * p.E + e;
        q[i] = p.part_p[at];
        d[i] = p.part_c[at];
      }
#pragma unroll
      for (int i = 0; i < B; ++i) {
        const bool in = u0 + 32 * i < count;
        sum += in ? (double)q[i] : 0.0;
        c += in ? d[i] : 0;
      }
    }
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) n += __shfl_xor(n, o, 64);
  if (lane == 0) sh_n[wave] = n;
  sh_p[i0][ie] = sum;
  sh_c[i0][ie] = c;
  __syncthreads();
  if (wave != 0) return;   // lanes of the upper half of wave 0 repeat the lower half's sums
  n = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) n += sh_n[i];
  sum = 0.0;
  c = 0;
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    sum += sh_p[i][ie];
    c += sh_c[i][ie];
  }
  const double inv_n = n > 0 ? 1.0 / n : 0.0;
  const double f = (double)c * p.E / p.topk * inv_n;
  const double scale = (double)p.coef / p.S;
  if (lane < kLossSlice && e < p.E) {
    p.counts[(int64_t)s * p.E + e] = c;
    p.dprob[(int64_t)s * p.E + e] = (float)(scale * f * inv_n);
  }
  const double part = group_sum_f64<64>(lane < kLossSlice && e < p.E ? f * sum * inv_n : 0.0);
  if (lane != 0) return;
  const unsigned slices = gridDim.x * gridDim.y;
  if (slices == 1) {
    *p.loss = (float)(scale * part);
    return;
  }
  auto add = [](uint64_t* at, uint64_t v) {
    return __hip_atomic_fetch_add(at, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  };
  uint64_t before = add(p.total, (uint64_t)(part / p.S * 0x1p53 + 0.5));
  asm volatile("s_waitcnt vmcnt(0)" : "+v"(before)::"memory");   // its value is here: the addition is done
  if (add(p.total + 1, 1) != slices - 1) return;
  *p.loss = (float)((double)p.coef * ((double)add(p.total, 0) * 0x1p-53));
}

// ---------------------------------------------------------------- backward
//
// With p the scores, ds the gradient reaching them:
//   softmax  dz = p (ds - sum p ds),    sigmoid  dz = (1 - p) (ds p), 1 - p = sigmoid(-z).
// What reaches the scores: the loss's dloss * dprob, on the normalised scores q (a
// sigmoid's are p / sum p: q (d - sum q d) takes the place of ds p), and at a chosen
// expert route_scale dw, or with renormalisation u (route_scale dw - sum over slots of
// route_scale dw u) in the place of ds p, u the normalised weights.
// Renormalised softmax weights do not depend on the other experts: their part of dz
// is added to the chosen experts as it is, so that the rounding of sum p ds, zero for
// it, does not reach the other experts' (the loss's) gradients, which are often far
// smaller.  A sigmoid's slots hold their part of dz too.
// The slots' values reach the lanes that hold their experts through one LDS row a
// token (the wave's own, so no barrier).

// A quotient's gradient u_i (x_i - sum u x), sum u = 1, does not change when one number is taken from every x.  Where one
// u is above a half, that x is taken: its own difference is then exactly 0, and what is left of a confident token, the
// others' u_j (x_j - x), is not the rounding of two nearly equal numbers (at 1 - u = 2^-24 nothing else was left).  With
// no u above a half nothing cancels, and 0 is taken.

// A product as it is rounded: fused into a difference from itself, it would leave its rounding there instead of 0.
__device__ __forceinline__ float rounded(float v) {
  asm("" : "+v"(v));
  return v;
}

// The x whose u is above a half, else 0 (in every lane of the token's group).
template <int LPT, int N>
__device__ __forceinline__ float dominant(const float (&u)[N], const float (&x)[N]) {
  float c = 0.0f;
#pragma unroll
  for (int v = 0; v < N; ++v) c += u[v] > 0.5f ? x[v] : 0.0f;
  return group_sum_f32<LPT>(c);
}

// A sigmoid token's sums for the loss's gradient where the scores' sum is below kSmallTotal, the only ones of which a score can
// hold more than half (a score is at most 1) or whose scores can be below the fp32 range: on the scale of the largest, and by
// differences from the dominant expert.  d: s (1 - s) on that scale; inv: one over the scores' sum on it; top and dot: the
// dominant expert's derivative and the mean of the differences from it.  Rare: the logits and the loss's derivative are read
// again, one at a time, through the token's LDS row `mine`, so that the kernel keeps its registers.
constexpr float kSmallTotal = 2.0f;
template <int LPT, int VPL, bool BF16, bool VEC>
__device__ __forceinline__ void small_sigmoid_sums(const void* __restrict__ logits, int64_t row,
                                                   const float* __restrict__ dprob, const float* __restrict__ dloss, int E,
                                                   int l, bool small, float* mine, float (&d)[VPL], float& inv, float& top,
                                                   float& dot) {
  const int n = small ? E : 0;
  const float dl = dloss != nullptr ? *dloss : 1.0f;
  float m = -kFltMax, total = 0.0f, most = 0.0f, of = 0.0f, sum = 0.0f;
#pragma unroll 1
  for (int v = 0; v < VPL; ++v) {
    const int e = expert_at<LPT, VEC>(l, v);
    if (e < n) m = fmaxf(m, gate_logit<BF16>(logits, row + e));
  }
  m = group_max_f32<LPT>(m);
  const float c = fminf(m, 0.0f);
#pragma unroll 1
  for (int v = 0; v < VPL; ++v) {
    const int e = expert_at<LPT, VEC>(l, v);
    if (e < n) {
      const float w = scaled_score<true>(gate_logit<BF16>(logits, row + e), c);   // 0 for -inf
      total += w;
      of = w > most ? rounded(dprob[e] * dl) : of;
      most = fmaxf(most, w);
    }
  }
  total = group_sum_f32<LPT>(total);
  const float x = group_sum_f32<LPT>(most > 0.5f * total ? of : 0.0f);
#pragma unroll 1
  for (int v = 0; v < VPL; ++v) {
    const int e = expert_at<LPT, VEC>(l, v);
    if (e < n) {
      const float z = gate_logit<BF16>(logits, row + e), w = scaled_score<true>(z, c);
      sum += w * (rounded(dprob[e] * dl) - x);
      mine[e] = w * sigmoid_parts(z).comp;
    } else {
      mine[e] = 0.0f;
    }
  }
  sum = group_sum_f32<LPT>(sum);
  wave_lds_fence();
  if (small) {
    inv = total > 0.0f && m >= kLeastSigmoid ? __fdiv_rn(1.0f, total) : 0.0f;
    top = x;
    dot = sum * inv;
#pragma unroll
    for (int v = 0; v < VPL; ++v) d[v] = mine[expert_at<LPT, VEC>(l, v)];
  }
  wave_lds_fence();
}

struct GateBwd {
  const void* logits;
  int64_t ld;
  int T, E, topk, renorm, chunk, S;
  const uint8_t* mask;
  float route_scale;
  const int32_t* ids;
  const float* dweights;   // null: the loss alone
  const int32_t* offs;
  const float* dprob;      // [S][E], null: the gate alone
  const float* dloss;      // null: 1
  void* dlogits;           // [T][E]
};

template <int LPT, int VPL, bool BF16, bool VEC, bool SIGMOID>
__global__ __launch_bounds__(256) void gate_bwd_kernel(GateBwd p) {
  constexpr int TPW = 64 / LPT, W = LPT * VPL;
  constexpr int KR = LPT == 64 ? 1 : 4;
  __shared__ __attribute__((aligned(16))) float s_row[256 * VPL];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l = lane % LPT, g = lane / LPT;
  float* const mine = s_row + (wave * TPW + g) * W;
  TokenRange rg;
  if (p.dprob != nullptr) {
    rg = gate_unit(p.offs, p.S, p.T, blockIdx.x, p.chunk);
  } else {
    const int64_t t0 = (int64_t)blockIdx.x * p.chunk;
    rg = TokenRange{-1, (int)min(t0, (int64_t)p.T), (int)min(t0 + p.chunk, (int64_t)p.T)};
  }
  float dp[VPL];   // the loss's gradient by the normalised scores
#pragma unroll
  for (int v = 0; v < VPL; ++v) dp[v] = 0.0f;
  if (rg.seq >= 0) {
    const float dl = p.dloss != nullptr ? *p.dloss : 1.0f;
    gate_load_vec<LPT, VPL, VEC>(p.dprob + (int64_t)rg.seq * p.E, p.E, l, dp);
#pragma unroll
    for (int v = 0; v < VPL; ++v) dp[v] = rounded(dp[v] * dl);
  }
  for (int base = rg.t0 + wave * TPW; base < rg.t1; base += 4 * TPW) {   // wave-uniform
    const int t = base + g;
    const bool live = t < rg.t1;
    const bool on = live && (p.mask == nullptr || p.mask[t] != 0);
    const int64_t row = (int64_t)t * p.ld, slot0 = (int64_t)t * p.topk;
    float z[VPL], s[VPL], ds[VPL], m, total;
    gate_load<LPT, VPL, BF16, VEC>(p.logits, row, p.E, l, on, z);
    int id[KR];
    float dw[KR];
    if (p.dweights != nullptr) {
#pragma unroll
      for (int r = 0; r < KR; ++r) {
        const int j = r * LPT + l;
        id[r] = on && j < p.topk ? p.ids[slot0 + j] : -1;
        if (id[r] < 0 || id[r] >= p.E) id[r] = -1;
        dw[r] = id[r] >= 0 ? rounded(p.dweights[slot0 + j] * p.route_scale) : 0.0f;
      }
    }
    float dot = 0.0f, top = 0.0f, inv;
    if constexpr (SIGMOID) {   // the loss's part, through the division by the scores' sum
      total = 0.0f;
#pragma unroll
      for (int v = 0; v < VPL; ++v) {
        const Sigmoid q = sigmoid_parts(z[v]);
        total += q.s;
        dot += dp[v] * q.s;
        ds[v] = q.slope;
      }
      total = group_sum_f32<LPT>(total);
      inv = total > 0.0f ? __fdiv_rn(1.0f, total) : 0.0f;
      dot = group_sum_f32<LPT>(dot) * inv;
      const bool small = rg.seq >= 0 && on && total < kSmallTotal;
      if (__ballot(small) != 0) {   // wave-uniform
        small_sigmoid_sums<LPT, VPL, BF16, VEC>(p.logits, row, p.dprob + (int64_t)rg.seq * p.E, p.dloss, p.E, l, small, mine, ds,
                                                inv, top, dot);
#pragma unroll
        for (int v = 0; v < VPL; ++v) ds[v] = ds[v] * inv * ((dp[v] - top) - dot);
      } else {
#pragma unroll
        for (int v = 0; v < VPL; ++v) ds[v] = ds[v] * inv * (dp[v] - dot);
      }
    } else {
      gate_scores<LPT, VPL, false>(z, s, m, total);   // all scores 0 when the token is off
      inv = total > 0.0f ? __fdiv_rn(1.0f, total) : 0.0f;
#pragma unroll
      for (int v = 0; v < VPL; ++v) {
        s[v] *= inv;
        ds[v] = dp[v];
      }
    }

    if (p.dweights != nullptr) {
      if (p.renorm) {
        float w[KR], comp[KR], ws = 0.0f, mean = 0.0f, c = -INFINITY;   // c: the lane's largest chosen logit
#pragma unroll
        for (int r = 0; r < KR; ++r) {
          w[r] = comp[r] = 0.0f;
          if (r * LPT >= p.topk) continue;   // uniform
          const float zj = id[r] >= 0 ? gate_logit<BF16>(p.logits, row + id[r]) : -INFINITY;
          if (!(zj > -INFINITY)) id[r] = -1, dw[r] = 0.0f;   // an ineligible expert passes nothing
          c = fmaxf(c, zj);
          if constexpr (SIGMOID) {
            const Sigmoid q = sigmoid_parts(zj);
            w[r] = q.s;
            comp[r] = q.comp;
          } else {
            w[r] = __expf(zj - m);
          }
          ws += w[r];
        }
        ws = group_sum_f32<LPT>(ws);
        if (__ballot(ws < kLowChosen && c > -INFINITY) != 0) {   // wave-uniform, rare: as the forward
          c = fmaxf(group_max_f32<LPT>(c), -kFltMax);
          if constexpr (SIGMOID) c = fminf(c, 0.0f);
          float scaled = 0.0f;
#pragma unroll
          for (int r = 0; r < KR; ++r) {
            const float zj = id[r] >= 0 ? gate_logit<BF16>(p.logits, row + id[r]) : -INFINITY;
            w[r] = ws < kLowChosen ? scaled_score<SIGMOID>(zj, c) : w[r];
            scaled += w[r];
          }
          ws = group_sum_f32<LPT>(scaled);
        }
#pragma unroll
        for (int r = 0; r < KR; ++r) w[r] = ws > 0.0f ? __fdiv_rn(w[r], ws) : 0.0f;
        const float first = dominant<LPT>(w, dw);
#pragma unroll
        for (int r = 0; r < KR; ++r) {
          dw[r] -= first;
          mean += dw[r] * w[r];
        }
        mean = group_sum_f32<LPT>(mean);
#pragma unroll
        for (int r = 0; r < KR; ++r) dw[r] = (dw[r] - mean) * w[r] * (SIGMOID ? comp[r] : 1.0f);
      } else if constexpr (SIGMOID) {
#pragma unroll
        for (int r = 0; r < KR; ++r)
          if (id[r] >= 0) {
            const float zj = gate_logit<BF16>(p.logits, row + id[r]);
            dw[r] *= sigmoid_parts(zj).slope;
            if (!(zj > -INFINITY)) id[r] = -1;   // an ineligible expert passes nothing
          }
      }
      // Slot values into the token's row.  Each slot first leaves its number at its expert: a slot that reads
      // another's shares its expert with it, and then the slots add up one after another, in their order.
#pragma unroll
      for (int v = 0; v < VPL; ++v) mine[expert_at<LPT, VEC>(l, v)] = 0.0f;
      wave_lds_fence();
#pragma unroll
      for (int r = 0; r < KR; ++r)
        if (id[r] >= 0) mine[id[r]] = (float)(r * LPT + l);
      wave_lds_fence();
      bool shared = false;
#pragma unroll
      for (int r = 0; r < KR; ++r)
        if (id[r] >= 0) shared = shared || mine[id[r]] != (float)(r * LPT + l);
      wave_lds_fence();
      if (__ballot(shared) == 0) {
#pragma unroll
        for (int r = 0; r < KR; ++r)
          if (id[r] >= 0) mine[id[r]] = dw[r];
      } else {
#pragma unroll
        for (int r = 0; r < KR; ++r)
          if (id[r] >= 0) mine[id[r]] = 0.0f;
        wave_lds_fence();
#pragma unroll
        for (int r = 0; r < KR; ++r)
          for (int j = 0; j < LPT; ++j) {
            if (r * LPT + j >= p.topk) break;   // uniform
            if (l == j && id[r] >= 0) mine[id[r]] += dw[r];
            wave_lds_fence();
          }
      }
      wave_lds_fence();
    }
    auto add_slots = [&] {
#pragma unroll
      for (int v = 0; v < VPL; ++v) ds[v] += mine[expert_at<LPT, VEC>(l, v)];
      wave_lds_fence();
    };
    const bool direct = SIGMOID || p.renorm;   // the slots hold their part of dz
    if (p.dweights != nullptr && !direct) add_slots();
    if (!on) {   // whatever the loss's gradient holds
#pragma unroll
      for (int v = 0; v < VPL; ++v) ds[v] = 0.0f;
    }
    if constexpr (!SIGMOID) {
      dot = 0.0f;
      if (__ballot(inv > 0.5f) != 0) {   // the largest softmax score is exp(0) inv; wave-uniform
        top = dominant<LPT>(s, ds);
#pragma unroll
        for (int v = 0; v < VPL; ++v) ds[v] -= top;
      }
#pragma unroll
      for (int v = 0; v < VPL; ++v) dot += s[v] * ds[v];
      dot = group_sum_f32<LPT>(dot);
#pragma unroll
      for (int v = 0; v < VPL; ++v) ds[v] = s[v] * (ds[v] - dot);
    }
    if (p.dweights != nullptr && direct) add_slots();
    // A score of 0 times an overflowed gradient is no 0: the ineligible experts' are set (wave-uniform, rare).
    if (__ballot(on && !(fabsf(dot) <= kFltMax)) != 0) {
#pragma unroll 1
      for (int v = 0; v < VPL; ++v) {
        const int e = expert_at<LPT, VEC>(l, v);
        mine[e] = e < (on ? p.E : 0) ? gate_logit<BF16>(p.logits, row + e) : -INFINITY;
      }
      wave_lds_fence();
#pragma unroll
      for (int v = 0; v < VPL; ++v) ds[v] = mine[expert_at<LPT, VEC>(l, v)] > -INFINITY ? ds[v] : 0.0f;
      wave_lds_fence();
    }
    if (live) {
      const int64_t out = (int64_t)t * p.E;
      if constexpr (VEC) {
#pragma unroll
        for (int c = 0; c < VPL / 4; ++c) {
          const int e0 = 4 * (l + LPT * c);
          if (e0 >= p.E) continue;
          if constexpr (BF16)
            *reinterpret_cast<u32x2*>(static_cast<__bf16*>(p.dlogits) + out + e0) =
                u32x2{__builtin_bit_cast(uint32_t, __builtin_convertvector(gt_f32x2{ds[4 * c], ds[4 * c + 1]}, gt_bf16x2)),
                      __builtin_bit_cast(uint32_t,
                                         __builtin_convertvector(gt_f32x2{ds[4 * c + 2], ds[4 * c + 3]}, gt_bf16x2))};
          else
            *reinterpret_cast<float4*>(static_cast<float*>(p.dlogits) + out + e0) =
                float4{ds[4 * c], ds[4 * c + 1], ds[4 * c + 2], ds[4 * c + 3]};
        }
      } else {
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
          const int e = expert_at<LPT, VEC>(l, v);
          if (e >= p.E) continue;
          if constexpr (BF16) static_cast<__bf16*>(p.dlogits)[out + e] = (__bf16)ds[v];
          else static_cast<float*>(p.dlogits)[out + e] = ds[v];
        }
      }
    }
  }
}

// ---------------------------------------------------------------- launchers

template <typename F>
static hipError_t gate_dispatch(int E, bool bf16, bool vec, bool sigmoid, F&& f) {
  using T = std::true_type;
  using N = std::false_type;
  auto types = [&](auto lpt, auto vpl) -> hipError_t {
    auto scored = [&](auto bf, auto ve) -> hipError_t {
      return sigmoid ? f(lpt, vpl, bf, ve, T{}) : f(lpt, vpl, bf, ve, N{});
    };
    if (bf16) return vec ? scored(T{}, T{}) : scored(T{}, N{});
    return vec ? scored(N{}, T{}) : scored(N{}, N{});
  };
  using std::integral_constant;
  // 16 lanes a token up to 256 experts, at most 16 logits a lane: lane steps are shared by the wave's tokens (65536 x 256:
  // a wave a token 120 us, 16 lanes 25 us).  Four lanes where they hold the logits in four registers; more logits on four
  // lanes, and 32 lanes for 257 to 512 experts, have not been measured.
  if (E <= 16) return types(integral_constant<int, 4>{}, integral_constant<int, 4>{});
  if (E <= 64) return types(integral_constant<int, 16>{}, integral_constant<int, 4>{});
  if (E <= 128) return types(integral_constant<int, 16>{}, integral_constant<int, 8>{});
  if (E <= 256) return types(integral_constant<int, 16>{}, integral_constant<int, 16>{});
  if (E <= 512) return types(integral_constant<int, 64>{}, integral_constant<int, 8>{});
  return types(integral_constant<int, 64>{}, integral_constant<int, 16>{});
}

static bool ptr_aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

hipError_t launch_moe_gate(const GateArgs& a, hipStream_t st) {
  const bool gate = a.gate, bal = a.loss != nullptr;
  GateFwd p;
  p.logits = a.logits;
  p.ld = a.ld;
  p.T = (int)a.tokens;
  p.E = a.E;
  p.topk = a.topk;
  p.renorm = a.renorm;
  p.chunk = bal ? gate_chunk(a.tokens, a.E) : gate_tile(a.tokens, a.E);
  p.S = a.S;
  const bool vec = a.E % 4 == 0 && a.ld % 4 == 0 && ptr_aligned(a.logits, a.bf16 ? 8 : 16) && ptr_aligned(a.bias, 16);
  p.bias = a.bias;
  p.mask = a.mask;
  p.route_scale = a.route_scale;
  p.ids = a.ids;
  p.weights = a.weights;
  p.offs = a.seq_offs;
  p.part_p = nullptr;
  p.part_c = nullptr;
  p.part_n = nullptr;
  p.total = nullptr;
  const int64_t units = bal ? gate_units(a.tokens, a.E, a.S) : (a.tokens + p.chunk - 1) / p.chunk;
  const int slices = (a.E + kLossSlice - 1) / kLossSlice;
  if (bal) {
    p.total = static_cast<uint64_t*>(a.workspace);
    p.part_p = reinterpret_cast<float*>(p.total + 2);
    p.part_c = reinterpret_cast<int32_t*>(p.part_p + units * a.E);
    p.part_n = p.part_c + units * a.E;
  }
  if (units > 0) {
    const hipError_t e = gate_dispatch(a.E, a.bf16, vec, a.sigmoid, [&](auto lpt, auto vpl, auto bf, auto ve, auto sg) -> hipError_t {
      constexpr int L = decltype(lpt)::value, V = decltype(vpl)::value;
      constexpr bool B = decltype(bf)::value, A = decltype(ve)::value, G = decltype(sg)::value;
      const dim3 grid((unsigned)units), block(256);
      if (gate && bal) hipLaunchKernelGGL((gate_kernel<L, V, B, A, G, true, true>), grid, block, 0, st, p);
      else if (gate) hipLaunchKernelGGL((gate_kernel<L, V, B, A, G, true, false>), grid, block, 0, st, p);
      else hipLaunchKernelGGL((gate_kernel<L, V, B, A, G, false, true>), grid, block, 0, st, p);
      return hipGetLastError();
    });
    if (e != hipSuccess) return e;
  }
  if (!bal) return hipSuccess;
  const GateLoss l{p.T,      p.E,      p.topk,   p.chunk, a.S,    a.coef,   a.seq_offs,
                   p.part_p, p.part_c, p.part_n, p.total, a.loss, a.counts, a.dprob};
  hipLaunchKernelGGL(gate_loss_kernel, dim3((unsigned)slices, (unsigned)a.S), dim3(1024), 0, st, l);
  return hipGetLastError();
}

hipError_t launch_moe_gate_backward(const GateBwdArgs& a, hipStream_t st) {
  if (a.tokens == 0) return hipSuccess;
  GateBwd p;
  p.logits = a.logits;
  p.ld = a.ld;
  p.T = (int)a.tokens;
  p.E = a.E;
  p.topk = a.topk;
  p.renorm = a.renorm;
  p.chunk = gate_chunk(a.tokens, a.E);
  p.S = a.S;
  const bool vec = a.E % 4 == 0 && a.ld % 4 == 0 && ptr_aligned(a.logits, a.bf16 ? 8 : 16) &&
                   ptr_aligned(a.dlogits, a.bf16 ? 8 : 16) && ptr_aligned(a.dprob, 16);
  p.mask = a.mask;
  p.route_scale = a.route_scale;
  p.ids = a.ids;
  p.dweights = a.dweights;
  p.offs = a.seq_offs;
  p.dprob = a.dprob;
  p.dloss = a.dloss;
  p.dlogits = a.dlogits;
  const int64_t units =
      a.dprob != nullptr ? gate_units(a.tokens, a.E, a.S) : (a.tokens + p.chunk - 1) / p.chunk;
  return gate_dispatch(a.E, a.bf16, vec, a.sigmoid, [&](auto lpt, auto vpl, auto bf, auto ve, auto sg) -> hipError_t {
    constexpr int L = decltype(lpt)::value, V = decltype(vpl)::value;
    constexpr bool B = decltype(bf)::value, A = decltype(ve)::value, G = decltype(sg)::value;
    hipLaunchKernelGGL((gate_bwd_kernel<L, V, B, A, G>), dim3((unsigned)units), dim3(256), 0, st, p);
    return hipGetLastError();
  });
}

}  // namespace fp8moe
