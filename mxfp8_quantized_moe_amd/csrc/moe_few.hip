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
// tile), the expert's tokens its columns, so one read of a tile serves up to 64 tokens; few_dot.hpp says how it is loaded.
// Codes become bf16 exactly (e4m3 and whole numbers up to 128 have at most eight significant bits); an e8m0 scale goes into
// that conversion, an fp32 scale divides the sum.  Activations come from L2 straight into registers.
//
// Tokens that choose one expert are found from the ids by every workgroup of the first kernel for itself (a
// token that names an expert twice is one column with the sum of its weights); workgroups behind the tiles' own leave the
// lists for the second kernel, which waits for nothing else: with a search by each of its waves 64 tokens of 32 experts took a
// fifth longer.
//
// Two kernels rather than one: the second needs all of a, so one kernel would hold a barrier over the GPU (not tried).
//
// Rates, the used experts' weights over the time of both kernels: 8 tokens of 16 experts, MX, 5120 x 8192: 115 us, 7 TB/s;
// 64 tokens of 32 experts 7168 x 2048, a quarter of their choices here: 215 us, 6.5 TB/s: bound by that read.  One token, six
// of 64 experts 2048 x 1408: 17 us, 3 TB/s, where the launches and the beginnings of the reads count as much.
#include "few_dot.hpp"
#include "kernels.hpp"
#include "swiglu_common.hpp"
#include "validate.hpp"

namespace fp8moe {

struct FewParams {
  const uint16_t* x;      // [T][ld_x]
  int64_t ld_x;
  const int32_t* ids;     // [T][topk]
  const float* weights;   // [T][topk]
  const uint8_t* w1;      // [E][2F][K]
  const uint8_t* w2;      // [E][K][F]
  const void* s1;
  const void* s2;
  uint16_t* y;            // [T][K]
  int T, topk, E, K, F;
  int ranks;              // experts that can be in use: min(E, T * topk)
  // workspace
  uint16_t* a2;           // [T * topk][F]: the row of a token's first slot of an expert
  float* part;            // [T * topk][K]: that slot's weighted product with W2
  int2* lists;            // [ranks][T]: an expert's tokens: token << 16 | slot, and the weight's bits
  int32_t* heads;         // [ranks]: id | tokens << 16
  int32_t* firsts;        // [T * topk]: 1 for a token's first slot of an expert, else 0
  int32_t* arrived;       // [ceil(K / 32)][32]: workgroups of the second kernel that are through with these columns
};

// ---------------------------------------------------------------- who chose whom

// LDS written by the wave's lanes so far is seen by its other lanes.
__device__ __forceinline__ void few_wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Every slot's expert (0xFFFF: none), a bitmap of the experts in use and their list.
struct FewIds {
  uint32_t bits[32];
  int n_act;
  uint16_t ids[kFewMaxSlots];
  uint16_t act[kFewMaxSlots];
};

// An expert's tokens in increasing order: token << 16 | the token's first slot of the expert, and its weight.
struct FewList {
  int ts[64];
  float w[64];
};

// The tokens of the expert of rank `rank`, by every wave for itself into its own list; their count (0: no expert of that
// rank).  How ranks are given out:
//  * up to 64 slots: in the order of the experts' first slots, a slot a lane, by ballots;
//  * no more experts than slots: rank and expert are the same, a token a lane;
//  * else through LDS, experts in increasing order (every thread of the workgroup calls it).
// The first two take no LDS and no barrier: a single token's 528 workgroups spent 3 of 16 us on those.
__device__ __forceinline__ int few_members(const FewParams& p, int rank, bool want_w, FewIds& s, FewList& l, int& e) {
  const int lane = threadIdx.x & 63, S = p.T * p.topk;
  bool first = false;
  int tok = lane, slot = 0;
  float w = 0.0f;
  if (S <= 64) {
    int id = lane < S ? p.ids[lane] : -1;
    if (id >= p.E) id = -1;
    unsigned long long rest = __ballot(id >= 0), m = 0;
    e = -1;
    for (int r = 0; rest != 0ull; ++r) {
      e = __builtin_amdgcn_readlane(id, __ffsll(rest) - 1);
      m = __ballot(id == e);
      if (r == rank) break;
      rest &= ~m;
    }
    if (rest == 0ull) return 0;
    if (id == e) {
      tok = lane / p.topk;
      slot = lane;
      unsigned long long own = m >> (tok * p.topk);           // the token's slots of this expert
      if (p.topk < 64) own &= (1ull << p.topk) - 1ull;
      first = (own & ((1ull << (lane - tok * p.topk)) - 1ull)) == 0ull;
      if (first && want_w)
        for (; own != 0ull; own &= own - 1ull) w += p.weights[tok * p.topk + __ffsll(own) - 1];
    }
  } else {
    if (p.E <= S) {
      e = rank;
      if (lane < p.T) {
        int at = -1;
#pragma unroll 8
        for (int j = p.topk - 1; j >= 0; --j) at = p.ids[lane * p.topk + j] == e ? j : at;
        first = at >= 0;
        slot = lane * p.topk + at;
      }
    } else {
      const int t = threadIdx.x;
      if (t < 32) s.bits[t] = 0;
      __syncthreads();
      for (int i = t; i < S; i += blockDim.x) {
        const int id = p.ids[i];
        const bool in = id >= 0 && id < p.E;
        s.ids[i] = in ? (uint16_t)id : (uint16_t)0xFFFF;
        if (in) atomicOr(&s.bits[id >> 5], 1u << (id & 31));
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
        for (at -= __popc(b); b != 0u; b &= b - 1u) s.act[at++] = (uint16_t)(32 * t + __ffs(b) - 1);
      }
      __syncthreads();
      if (rank >= s.n_act) return 0;
      e = s.act[rank];
      if (lane < p.T) {
        int at = -1;
        for (int j = p.topk - 1; j >= 0; --j) at = (int)s.ids[lane * p.topk + j] == e ? j : at;
        first = at >= 0;
        slot = lane * p.topk + at;
      }
    }
    if (first && want_w)
      for (int j = slot; j < (lane + 1) * p.topk; ++j)
        if (p.ids[j] == e) w += p.weights[j];
  }
  e = __builtin_amdgcn_readfirstlane(e);
  const unsigned long long m = __ballot(first);
  if (first) {
    const int at = __popcll(m & ((1ull << lane) - 1ull));
    l.ts[at] = (tok << 16) | slot;
    l.w[at] = w;
  }
  few_wave_sync();
  return __popcll(m);
}

// ---------------------------------------------------------------- the two kernels

// Sixteen bytes to memory past the XCD's caches, as a relaxed atomic store at agent scope would go, in one piece.  The
// registers of such a wide store may be written again two wait states later, which the compiler, blind to what the
// block does, would not keep.
__device__ __forceinline__ void few_store_agent16(float* to, few_v4f v) {
  asm volatile("global_store_dwordx4 %0, %1, off sc1\n\ts_nop 1" ::"v"(to), "v"(v) : "memory");
}

// A workgroup takes NT (2 or 4) tiles of 16 weight rows of one expert for all its tokens; its W waves split the
// contraction and add up through LDS.
//
// UP: gate rows and the matching up rows of W1; writes 8 NT columns of a = silu(g) * u.  Behind the
// tiles' workgroups one for each rank writes the expert's list for the second kernel, and one more the counters
// and the slots' marks.
//
// Else 16 NT rows of W2: as many columns of each token's product, times its weight, go to the slot's row of `part`; the
// last workgroup that is through with these columns adds up each token's slots in order and writes y.  Rows of part
// are written and read past the caches of an XCD (agent scope), and a workgroup's stores have reached memory before
// it counts itself, each column range on a cache line of its own; which one is last changes nothing.
template <int FMT, bool UP, int W, int NT, bool STREAM>
__global__ __launch_bounds__(64 * W) void few_kernel(FewParams p) {
  constexpr int PAIRS = NT / 2, COLS = UP ? 16 * PAIRS : 16 * NT;   // columns of the result
  __shared__ few_v4f red[W][4 * NT][64];
  __shared__ FewIds ids;
  __shared__ FewList lists[W];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int N = UP ? p.F : p.K, tiles = (N + COLS - 1) / COLS;
  const int rank = blockIdx.x / tiles, tile = blockIdx.x - rank * tiles;
  const int L = UP ? p.K : p.F;
  FewList& list = lists[wave];
  int e, n;
  if constexpr (UP) {
    if (rank >= p.ranks) {
      const int r = blockIdx.x - p.ranks * tiles;
      if (r < p.ranks) {
        n = few_members(p, r, true, ids, list, e);
        if (wave == 0) {
          if (lane == 0) p.heads[r] = n > 0 ? e | (n << 16) : 0;
          if (lane < n) p.lists[r * p.T + lane] = int2{list.ts[lane], __float_as_int(list.w[lane])};
        }
        return;
      }
      for (int i = threadIdx.x; i < (p.K + 31) / 32; i += 64 * W) p.arrived[32 * i] = 0;
      const int S = p.T * p.topk;
      for (int i = threadIdx.x; i < S; i += 64 * W) {
        const int id = p.ids[i];
        ids.ids[i] = id >= 0 && id < p.E ? (uint16_t)id : (uint16_t)0xFFFF;
      }
      __syncthreads();
      for (int i = threadIdx.x; i < S; i += 64 * W) {
        bool f = ids.ids[i] != 0xFFFF;
        for (int j = i - i % p.topk; j < i; ++j) f &= ids.ids[j] != ids.ids[i];
        p.firsts[i] = f;
      }
      return;
    }
    n = few_members(p, rank, false, ids, list, e);
    if (n == 0) return;
  } else {
    const int head = __builtin_amdgcn_readfirstlane(p.heads[rank]);
    e = head & 0xFFFF;
    n = head >> 16;
    const int2 v = p.lists[rank * p.T + min(lane, p.T - 1)];
    list.ts[lane] = v.x;
    list.w[lane] = __int_as_float(v.y);
    few_wave_sync();
  }
  if (UP || n > 0) {
    const int64_t row0 = (int64_t)e * (UP ? 2 * p.F : p.K);   // the expert's first weight row
    const int64_t rows = (int64_t)p.E * (UP ? 2 * p.F : p.K);
    const uint8_t* const wp = UP ? p.w1 : p.w2;
    const void* const sp = UP ? p.s1 : p.s2;
    // a lane will write four columns of each tile: c .. c + 3
    const int c = 4 * (lane >> 4);
    FewTile w[NT];
    few_v4f div[NT];
#pragma unroll
    for (int h = 0; h < NT; ++h) {
      // tile h's first row in the expert; a tile behind the last one is the first again, and not written
      const int col = UP ? 16 * (tile * PAIRS + h / 2) : 16 * (tile * NT + h);
      const int64_t row = row0 + (col < N ? col : 0) + (UP && (h & 1) ? p.F : 0);
      w[h] = few_tile<FMT>(wp, sp, row, rows, L);
      div[h] = few_v4f{1.0f, 1.0f, 1.0f, 1.0f};
      if constexpr (FMT == kFewFp8 || FMT == kFewInt8)
        div[h] = *reinterpret_cast<const few_f4u*>(static_cast<const float*>(sp) + row + c);
    }
    few_blocks<NT>(n, [&](auto nb_tag, auto q_tag) {
      constexpr int NB = decltype(nb_tag)::value, Q = decltype(q_tag)::value;
      using Dot = FewDot<FMT, NT, NB, Q, STREAM>;
      uint32_t x[NB];
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int ts = list.ts[min(Dot::ROWS * b + Dot::slot_of(lane), n - 1)];
        x[b] = UP ? (uint32_t)(2 * (ts >> 16) * p.ld_x) : (uint32_t)(2 * (ts & 0xFFFF) * p.F);
      }
      Dot d;
      d.run(w, UP ? p.x : p.a2, x, L, wave, W);
#pragma unroll
      for (int h = 0; h < NT; ++h)
#pragma unroll
        for (int b = 0; b < NB; ++b) red[wave][h * NB + b][lane] = d.sums(h, b);
      __syncthreads();
      // a lane takes token 16 i + (l & 15), columns 4 (l >> 4) .. + 3 of the tiles, two tiles at a time
      for (int i = wave; i < (NB * Dot::ROWS + 15) / 16 * PAIRS; i += W) {
        const int m = 16 * (i / PAIRS) + (lane & 15), b = m / Dot::ROWS;
        const int col = 16 * (UP ? 1 : 2) * (tile * PAIRS + i % PAIRS);   // first column of the pair
        if (m >= n || col >= N) continue;
        few_v4f g = {0.0f, 0.0f, 0.0f, 0.0f}, u = g, dg = div[0], du = div[1];
        if constexpr (PAIRS > 1) {
          if (i % PAIRS) dg = div[2], du = div[3];
        }
#pragma unroll
        for (int v = 0; v < W; ++v) {
          const int from = 16 * (lane >> 4) + Q * (m % Dot::ROWS);
          g += red[v][2 * (i % PAIRS) * NB + b][from];
          u += red[v][(2 * (i % PAIRS) + 1) * NB + b][from];
        }
        const int slot = list.ts[m] & 0xFFFF;
        if constexpr (UP) {
          float a[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float gj = __fdiv_rn(g[j], dg[j]), uj = __fdiv_rn(u[j], du[j]);
            a[j] = gj * sw_sigmoid(gj) * uj;
          }
          *reinterpret_cast<u32x2*>(p.a2 + (int64_t)slot * p.F + col + c) = u32x2{sw_pack(a[0], a[1]), sw_pack(a[2], a[3])};
        } else {
          float* o = p.part + (int64_t)slot * p.K + col + c;
          const float wt = list.w[m];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            g[j] = wt * __fdiv_rn(g[j], dg[j]);
            u[j] = wt * __fdiv_rn(u[j], du[j]);
          }
          few_store_agent16(o, g);
          if (col + 16 < N) few_store_agent16(o + 16, u);
        }
      }
    });
  }
  if constexpr (!UP) {
    __shared__ int s_last;
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // this wave's stores have reached memory
    __syncthreads();
    if (threadIdx.x == 0)
      s_last = __hip_atomic_fetch_add(p.arrived + 32 * tile, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == p.ranks - 1;
    __syncthreads();
    if (!s_last) return;
    // two columns a thread: four bytes of y
    for (int i = threadIdx.x; i < p.T * (COLS / 2); i += 64 * W) {
      const int t = i / (COLS / 2), col = tile * COLS + 2 * (i % (COLS / 2));
      if (col >= p.K) continue;
      float a = 0.0f, b = 0.0f;
#pragma unroll 8
      for (int j = 0; j < p.topk; ++j) {
        const int slot = t * p.topk + j;
        const unsigned long long v = __hip_atomic_load(reinterpret_cast<const unsigned long long*>(p.part + (int64_t)slot * p.K + col),
                                                       __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        const bool f = p.firsts[slot] != 0;   // other slots' rows hold nothing
        a += f ? __uint_as_float((uint32_t)v) : 0.0f;
        b += f ? __uint_as_float((uint32_t)(v >> 32)) : 0.0f;
      }
      *reinterpret_cast<uint32_t*>(p.y + (int64_t)t * p.K + col) = sw_pack(a, b);
    }
  }
}

// Without F there is no product: y is zero.
__global__ __launch_bounds__(256) void few_zero_kernel(uint32_t* y, int64_t n) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i < n) y[i] = 0;
}

template <int FMT, bool UP>
static hipError_t few_launch(const FewParams& p, hipStream_t st) {
  // Four tiles a workgroup share the activations' loads, which outgrow the weights' where experts have some 25 tokens (up to
  // 32 two tiles load whole cache lines of them), if the workgroups still fill the GPU (64 tokens, eight of 16 experts
  // 5120 x 8192: both kernels 669 -> 585 us by the first, -> 643 by the second; eight of 8 7168 x 2048 191 -> 153, -> 174; six
  // of 16 2048 x 1408, 24 an expert, 64.6 -> 65.1, -> 61.7; 64 tokens of one expert 4096 x 8192, the second's 64 workgroups:
  // 69 -> 90; four tokens an expert of 32, 7168 x 2048, the others' ids none: both 231 -> 249). The host knows the choices, not
  // how many of them name an expert here.
  auto count = [&](int cols) { return (int64_t)p.ranks * (((UP ? p.F : p.K) + cols - 1) / cols); };
  constexpr int COLS = UP ? 16 : 32;
  const bool wide = (int64_t)p.T * p.topk >= 24 * (int64_t)p.E && count(2 * COLS) >= 224;
  const int64_t blocks = count(wide ? 2 * COLS : COLS);
  const dim3 grid((unsigned)(blocks + (UP ? p.ranks + 1 : 0)));
  // Short rows leave four waves a step or two each: two waves where the workgroups fill the GPU by themselves
  // (64 tokens of 64 experts 2048 x 1408: first kernel 75 -> 68 us; rows of 7168: 149 -> 154 us).
  const bool two = !wide && (UP ? p.K : p.F) <= 2048 && blocks >= 512;
  // Streamed loads where the experts' weights are beyond the last-level cache (64 tokens of 32 experts 7168 x 2048, 1.4 GB:
  // first kernel 153 -> 144 us); smaller ones are not, which may stay there from one call to the next (4 tokens of 7 experts
  // 1040 x 336, 7 MB: 11.9 us streamed, 5.8 not; 5 tokens of them, weights from HBM: 16.5 and 11.6, both kernels).
  const bool stream = (int64_t)p.E * 3 * p.K * p.F > (256ll << 20);
  auto kern = wide ? few_kernel<FMT, UP, 4, 4, false>
              : stream ? (two ? few_kernel<FMT, UP, 2, 2, true> : few_kernel<FMT, UP, 4, 2, true>)
                       : (two ? few_kernel<FMT, UP, 2, 2, false> : few_kernel<FMT, UP, 4, 2, false>);
  hipLaunchKernelGGL(kern, grid, dim3(two ? 128 : 256), 0, st, p);
  return hipGetLastError();
}

template <int FMT>
static hipError_t few_both(const FewParams& p, hipStream_t st) {
  const hipError_t err = few_launch<FMT, true>(p, st);
  return err != hipSuccess ? err : few_launch<FMT, false>(p, st);
}

hipError_t launch_moe_few_tokens(const FewArgs& a, hipStream_t st) {
  if (a.tokens == 0 || a.K == 0) return hipSuccess;
  if (a.F == 0) {
    const int64_t n = a.tokens * a.K / 2;
    hipLaunchKernelGGL(few_zero_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, st, reinterpret_cast<uint32_t*>(a.y), n);
    return hipGetLastError();
  }
  FewParams p{a.x, a.ld_x, a.ids, a.weights, a.w1, a.w2, a.s1, a.s2, a.y,
              (int)a.tokens, a.topk, a.n_experts, (int)a.K, (int)a.F};
  const int64_t slots = a.tokens * a.topk;
  p.ranks = (int)std::min<int64_t>(slots, a.n_experts);
  char* ws = static_cast<char*>(a.workspace);   // few_workspace_bytes, in this order (each part's size keeps the next aligned)
  auto take = [&](int64_t bytes) {
    char* at = ws;
    ws += bytes;
    return at;
  };
  p.a2 = reinterpret_cast<uint16_t*>(take(slots * a.F * 2));
  p.part = reinterpret_cast<float*>(take(slots * a.K * 4));
  p.lists = reinterpret_cast<int2*>(take(slots * a.tokens * 8));
  p.heads = reinterpret_cast<int32_t*>(take(slots * 4));
  p.firsts = reinterpret_cast<int32_t*>(take(slots * 4));
  p.arrived = reinterpret_cast<int32_t*>(take((a.K + 31) / 32 * 128));
  switch (a.fmt) {
    case kFewFp8: return few_both<kFewFp8>(p, st);
    case kFewInt8: return few_both<kFewInt8>(p, st);
    case kFewMx: return few_both<kFewMx>(p, st);
    default: return few_both<kFewMxK4>(p, st);
  }
}

}  // namespace fp8moe
