// The integer grouped GEMM for few rows a group (a decoding step): out[m][n] =
// (sum over k of a[m][k] b[e][n][k]) / (sa[m] sb[e][n]) for the rows m of group e.
//
// With few rows the product is the read of the groups' weights. The persistent GEMM's
// 256-column tiles are too few then to ask memory for enough at once (16 rows of 14336
// columns of 4096: 56 workgroups on 256 CUs, 37 us; the weights at the copy rate take 11), so a
// workgroup here takes 32 or 64 columns for up to 64 rows (12 us), its waves split the
// contraction, and the whole-number sums are added up through LDS. Sums are exact in any order and the
// epilogue's operations are the persistent GEMM's, so both give the same bits.
#include "few_dot.hpp"
#include "kernels.hpp"

namespace fp8moe {

namespace {

constexpr int kUnitRows = 64;   // rows of a group that share a read of the weights

struct I8Params {
  const uint8_t* a;
  const uint8_t* b;
  const float* sa;
  const float* sb;
  const int32_t* offs;
  void* out;
  int E, M, N, K;
};

struct UnitChunks {
  __device__ int operator()(int lo, int hi) const { return (hi - lo + kUnitRows - 1) / kUnitRows; }
};
struct NoPad {
  __device__ int operator()(int, int) const { return 0; }
};

template <int OUT, int W, int NT, bool STREAM>
__global__ __launch_bounds__(64 * W) void i8_rows_kernel(I8Params p) {
  __shared__ few_v4i red[W][4 * NT][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  constexpr int COLS = 16 * NT;
  const int tiles = (p.N + COLS - 1) / COLS;
  const int unit = blockIdx.x / tiles, tile = blockIdx.x - unit * tiles;
  const Unit un = find_unit_quant<64 * W>(p.offs, p.E, p.M, unit, UnitChunks{}, NoPad{});
  if (un.e < 0) return;
  const int e = __builtin_amdgcn_readfirstlane(un.e);
  const int m0 = __builtin_amdgcn_readfirstlane(un.lo + un.j * kUnitRows);
  const int n = min(kUnitRows, __builtin_amdgcn_readfirstlane(un.hi) - m0);
  // A tile that N ends in starts earlier and leaves out the columns before `cn`; where N is below the tile's width (it is
  // 16 or more) its later sixteens do.
  const int cn = tile * COLS, c0 = max(0, min(cn, p.N - COLS));
  const int64_t row = (int64_t)e * p.N + c0, rows = (int64_t)p.E * p.N;
  int c[NT];   // of its h-th sixteen a lane writes columns c[h] .. c[h] + 3
  FewTile w[NT];
  few_f4u sq[NT];
#pragma unroll
  for (int h = 0; h < NT; ++h) {
    const int off = min(16 * h, p.N - c0 - 16);
    c[h] = c0 + off + 4 * (lane >> 4);
    w[h] = few_tile<kFewInt8Both>(p.b, nullptr, row + off, rows, p.K);
    sq[h] = *reinterpret_cast<const few_f4u*>(p.sb + row + off + 4 * (lane >> 4));
  }
  few_blocks<NT>(n, [&](auto nb_tag, auto q_tag) {
    constexpr int NB = decltype(nb_tag)::value, Q = decltype(q_tag)::value;
    using Dot = FewDot<kFewInt8Both, NT, NB, Q, STREAM>;
    uint32_t x[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) x[b] = (uint32_t)(min(Dot::ROWS * b + Dot::slot_of(lane), n - 1) * p.K);
    Dot d;
    d.run(w, p.a + (int64_t)m0 * p.K, x, p.K, wave, W);
#pragma unroll
    for (int h = 0; h < NT; ++h)
#pragma unroll
      for (int b = 0; b < NB; ++b) red[wave][h * NB + b][lane] = d.sums(h, b);
    __syncthreads();
    for (int i = wave; i < (NB * Dot::ROWS + 15) / 16; i += W) {
      const int m = 16 * i + (lane & 15), b = m / Dot::ROWS;
      if (m >= n) continue;
      const float sp = p.sa[m0 + m], inv_p = __frcp_rn(sp);
#pragma unroll
      for (int h = 0; h < NT; ++h) {
        few_v4i s = {0, 0, 0, 0};
#pragma unroll
        for (int v = 0; v < W; ++v) s += red[v][h * NB + b][16 * (lane >> 4) + Q * (m % Dot::ROWS)];
        float o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float inv_q = __frcp_rn(sq[h][j]);
          if constexpr (OUT == 0) o[j] = (float)s[j] * inv_p * inv_q;
          else o[j] = div_both((float)s[j], sp, inv_p, sq[h][j], inv_q);
        }
        const int col = c[h], first = max(cn, c0 + 16 * h);
        const int64_t at = (int64_t)(m0 + m) * p.N + col;
        if ((p.N * (OUT == 0 ? 2 : 4)) % 16 == 0) {   // then c0 and `first` are multiples of four
          if (col < first) continue;
          if constexpr (OUT == 0)
            *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(p.out) + at) = u32x2{few_pack(o[0], o[1]), few_pack(o[2], o[3])};
          else
            *reinterpret_cast<few_v4f*>(static_cast<float*>(p.out) + at) = few_v4f{o[0], o[1], o[2], o[3]};
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (col + j < first) continue;
            if constexpr (OUT == 0) static_cast<__bf16*>(p.out)[at + j] = (__bf16)o[j];
            else static_cast<float*>(p.out)[at + j] = o[j];
          }
        }
      }
    }
  });
}

}  // namespace

// When this kernel is taken, by the persistent GEMM's tiles of 256 columns (one for each group with rows). They fill the
// GPU: up to 16 rows a group (64 groups, 2816 x 2048: 512 rows of 1408 37 us here, 44 there; 1024 rows 70 and 72; 1500 rows 76
// and 73; 1000 rows of 32 groups 53 and 45). They do not: their time is one pass along K whatever the rows are, while the
// activations' loads here grow with them (one group of 14336 x 4096: 16 rows 12 and 40 us, 256 rows 40 and 46; 4096 x 4096: 400
// rows 22 and 45, 1024 rows 44 and 45; 4000 of 1024 x 1024 14 and 20; 2048 rows in 8 groups of 1024 x 2048 18 and 19; 447 of
// 10756 x 1024 27 and 22).
bool i8_rows_wanted(const GemmArgs& g) {
  if (g.N < 16) return false;
  const int64_t groups = std::min<int64_t>(g.n_groups, g.M);
  if ((g.M / kUnitRows + groups) * ((g.N + 31) / 32) >= 1 << 24) return false;   // a launch takes fewer than 2^32 threads
  return g.M <= 16 * (int64_t)g.n_groups ||
         (groups * ((g.N + 255) / 256) < 256 && (g.M + 64 * groups) * g.N <= 4600000);
}

template <int NT>
static hipError_t i8_rows(const GemmArgs& g, hipStream_t st) {
  const I8Params p{static_cast<const uint8_t*>(g.a), static_cast<const uint8_t*>(g.b), static_cast<const float*>(g.sa),
                   static_cast<const float*>(g.sb), g.offs, g.out, g.n_groups, (int)g.M, (int)g.N, (int)g.K};
  const int64_t blocks = (g.M / kUnitRows + std::min<int64_t>(g.n_groups, g.M)) * ((g.N + 16 * NT - 1) / (16 * NT));
  const bool two = g.K <= 2048 && blocks >= 512;
  const bool stream = (int64_t)g.n_groups * g.N * g.K > (256ll << 20);
  auto pick = [&](auto out_tag) {
    constexpr int OUT = decltype(out_tag)::value;
    if constexpr (NT == 2) {
      if (stream && two) return i8_rows_kernel<OUT, 2, NT, true>;
    }   // wider tiles have (M + 64 groups) * N <= 4600000 and M > 32 groups, so streamed rows are longer than 5600
    return stream ? i8_rows_kernel<OUT, 4, NT, true> : two ? i8_rows_kernel<OUT, 2, NT, false> : i8_rows_kernel<OUT, 4, NT, false>;
  };
  auto kern = g.out_dtype == 0 ? pick(std::integral_constant<int, 0>{}) : pick(std::integral_constant<int, 1>{});
  hipLaunchKernelGGL(kern, dim3((unsigned)blocks), dim3(two ? 128 : 256), 0, st, p);
  return hipGetLastError();
}

hipError_t launch_i8_rows(const GemmArgs& g, hipStream_t st) {
  // Wider tiles share the activations' loads: 64 columns for more than 32 rows a group where their workgroups fill the GPU
  // (128 rows of 14336 x 4096 34 -> 23 us, 1000 of 1024 x 4096 17 -> 15; 128 of 4096 12.6 -> 14.5, 700 rows in 32 groups of
  // 7168 x 2048 90 -> 103).
  const int64_t groups = std::min<int64_t>(g.n_groups, g.M);
  return g.N >= 64 && g.M > 32 * groups && (g.M / kUnitRows + groups) * ((g.N + 63) / 64) >= 224 ? i8_rows<4>(g, st)
                                                                                                  : i8_rows<2>(g, st);
}

}  // namespace fp8moe
