// The integer grouped GEMM for few rows a group (a decoding step): out[m][n] =
// (sum over k of a[m][k] b[e][n][k]) / (sa[m] sb[e][n]) for the rows m of group e.
//
// With few rows the product is the read of the groups' weights. The persistent GEMM's
// 256-column tiles are too few then to ask memory for enough at once (16 rows of 14336
// columns of 4096: 56 workgroups on 256 CUs, 37 us; the weights at the copy rate take 11), so a
// workgroup here takes 32 or 64 columns for up to 64 rows (14.6 us), its waves split the
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
  // a tile that N ends in starts earlier and leaves out the columns before `cn`
  const int cn = tile * COLS, c0 = min(cn, p.N - COLS);
  const int64_t row = (int64_t)e * p.N + c0, rows = (int64_t)p.E * p.N;
  const int c = c0 + 4 * (lane >> 4);   // a lane writes columns c .. c + 3 of each tile of 16
  FewTile w[NT];
  few_f4u sq[NT];
#pragma unroll
  for (int h = 0; h < NT; ++h) {
    w[h] = few_tile<kFewInt8Both>(p.b, nullptr, row + 16 * h, rows, p.K);
    sq[h] = *reinterpret_cast<const few_f4u*>(p.sb + row + 16 * h + 4 * (lane >> 4));
  }
  few_blocks<NT>(n, [&](auto nb_tag, auto q_tag) {
    constexpr int NB = decltype(nb_tag)::value, Q = decltype(q_tag)::value;
    using Dot = FewDot<kFewInt8Both, NT, NB, Q, STREAM>;
    uint32_t x[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) x[b] = (uint32_t)(min(Dot::ROWS * b + (lane & 15) % Dot::ROWS, n - 1) * p.K);
    const int steps = (p.K + Dot::STEP - 1) / Dot::STEP;
    Dot d;
    d.run(w, p.a + (int64_t)m0 * p.K, x, p.K, steps * wave / W, steps * (wave + 1) / W);
#pragma unroll
    for (int r = 0; r < Dot::R; ++r)
#pragma unroll
      for (int b = 0; b < NB; ++b) red[wave][r * NB + b][lane] = d.acc[r][b];
    __syncthreads();
    for (int i = wave; i < (NB * Dot::ROWS + 15) / 16; i += W) {
      const int m = 16 * i + (lane & 15), cq = lane >> 4, b = m / Dot::ROWS;
      if (m >= n) continue;
      const float inv_p = __frcp_rn(p.sa[m0 + m]);
#pragma unroll
      for (int h = 0; h < NT; ++h) {
        few_v4i s = {0, 0, 0, 0};
#pragma unroll
        for (int v = 0; v < W; ++v)
#pragma unroll
          for (int q = 0; q < Q; ++q)
            s += red[v][(h * Q + cq / (4 / Q)) * NB + b][Dot::lane_of(cq, m % Dot::ROWS, q)];
        float o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = (float)s[j] * inv_p * __frcp_rn(sq[h][j]);
        const int col = c + 16 * h;
        const int64_t at = (int64_t)(m0 + m) * p.N + col;
        if ((p.N * (OUT == 0 ? 2 : 4)) % 16 == 0) {   // then cn - c0 is a multiple of four
          if (col < cn) continue;
          if constexpr (OUT == 0)
            *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(p.out) + at) = u32x2{few_pack(o[0], o[1]), few_pack(o[2], o[3])};
          else
            *reinterpret_cast<few_v4f*>(static_cast<float*>(p.out) + at) = few_v4f{o[0], o[1], o[2], o[3]};
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (col + j < cn) continue;
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
// GPU: up to eight rows a group (64 groups, 2816 x 2048: 384 rows 60 us here, 72 there; 1024 rows 81 and 72). They do not:
// their time is one pass along K whatever the rows are, while the activations' loads here grow with them (14336 x 4096,
// one group: 16 rows 14.6 and 37 us, 128 rows 34 and 40, 192 rows 49 and 46; 200 rows of 4096 x 1024 8.5 and 20; 509 rows in
// 11 groups of 1999 x 2064 20 and 26).
bool i8_rows_wanted(const GemmArgs& g) {
  if (g.N < 32) return false;
  const int64_t groups = std::min<int64_t>(g.n_groups, g.M);
  return g.M <= 8 * (int64_t)g.n_groups || (groups * ((g.N + 255) / 256) < 256 && (g.M + 64 * groups) * g.N <= 3000000);
}

template <int NT>
static hipError_t i8_rows(const GemmArgs& g, hipStream_t st) {
  const I8Params p{static_cast<const uint8_t*>(g.a), static_cast<const uint8_t*>(g.b), static_cast<const float*>(g.sa),
                   static_cast<const float*>(g.sb), g.offs, g.out, g.n_groups, (int)g.M, (int)g.N, (int)g.K};
  const int64_t blocks = (g.M / kUnitRows + std::min<int64_t>(g.n_groups, g.M)) * ((g.N + 16 * NT - 1) / (16 * NT));
  if (blocks > 0x7FFFFFFF) return hipErrorInvalidValue;
  const bool two = g.K <= 2048 && blocks >= 512;
  const bool stream = (int64_t)g.n_groups * g.N * g.K > (256ll << 20);
  auto pick = [&](auto out_tag) {
    constexpr int OUT = decltype(out_tag)::value;
    return stream ? (two ? i8_rows_kernel<OUT, 2, NT, true> : i8_rows_kernel<OUT, 4, NT, true>)
                  : (two ? i8_rows_kernel<OUT, 2, NT, false> : i8_rows_kernel<OUT, 4, NT, false>);
  };
  auto kern = g.out_dtype == 0 ? pick(std::integral_constant<int, 0>{}) : pick(std::integral_constant<int, 1>{});
  hipLaunchKernelGGL(kern, dim3((unsigned)blocks), dim3(two ? 128 : 256), 0, st, p);
  return hipGetLastError();
}

hipError_t launch_i8_rows(const GemmArgs& g, hipStream_t st) {
  // Wider tiles share the activations' loads: 64 columns for more than 16 rows a group (64 rows of 14336 x 4096 25 -> 20 us;
  // 4 rows 12.8 -> 15).
  return g.N >= 64 && g.M > 16 * std::min<int64_t>(g.n_groups, g.M) ? i8_rows<4>(g, st) : i8_rows<2>(g, st);
}

}  // namespace fp8moe
