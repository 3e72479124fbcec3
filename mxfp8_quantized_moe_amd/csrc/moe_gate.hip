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
// Selection works on 64-bit keys: a double holds an fp32 logit exactly, and its low
// ten bits, which the key does not need, hold the expert's index (complemented for
// positive keys), so one maximum finds the winner and breaks ties to the lower
// index.  With a bias the key is the score plus the bias in 64 bits: scores next to
// each other would otherwise be ordered by fp32 rounding.
//
// One wave takes one token; lane l holds experts l, l + 64, ...
#include "device_common.hpp"
#include "kernels.hpp"
#include "validate.hpp"

namespace fp8moe {

static_assert(kGateMaxExperts == 1024, "ten bits of a key hold the index, a wave holds 16 logits a lane");

constexpr float kFltMax = 3.402823466e38f;

// ---------------------------------------------------------------- wave helpers

__device__ __forceinline__ float gate_max(float v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor(v, o, 64));
  return v;
}
__device__ __forceinline__ float gate_sum(float v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}
__device__ __forceinline__ double gate_sum(double v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}
__device__ __forceinline__ double gate_max(double v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v = fmax(v, __shfl_xor(v, o, 64));
  return v;
}

// The logit as the gate reads it: NaN as -inf, at most the largest finite value.
template <bool BF16>
__device__ __forceinline__ float gate_logit(const void* __restrict__ logits, int64_t at) {
  float v;
  if constexpr (BF16) v = __uint_as_float((uint32_t)static_cast<const uint16_t*>(logits)[at] << 16);
  else v = static_cast<const float*>(logits)[at];
  return v != v ? -INFINITY : fminf(v, kFltMax);
}

// key with the index in its low ten bits; -inf stays as it is (no expert to name).
__device__ __forceinline__ double gate_pack(double key, int idx) {
  if (!(key > -INFINITY)) return -INFINITY;
  const int64_t b = __double_as_longlong(fmin(fmax(key, -1.7e308), 1.7e308) + 0.0);   // -0 -> +0
  return __longlong_as_double((b & ~1023ll) | (b >= 0 ? 1023 - idx : idx));
}
__device__ __forceinline__ int gate_index(double key) {
  const int64_t b = __double_as_longlong(key);
  return (int)(b >= 0 ? 1023 - (b & 1023) : (b & 1023));
}

__device__ __forceinline__ float sigmoid_f32(float z) { return __builtin_amdgcn_rcpf(1.0f + __expf(-z)); }

// ---------------------------------------------------------------- work units
//
// A workgroup takes one unit: up to `chunk` tokens of one sequence (or of the
// tokens behind the last one).  Without the loss there is one sequence of all.

struct TokenRange {
  int seq;      // -1: behind the last sequence (or past the end)
  int t0, t1;
};
__device__ __forceinline__ TokenRange gate_unit(const int32_t* __restrict__ offs, int S, int T, int u, int chunk) {
  auto chunks = [chunk](int lo, int hi) { return (hi - lo + chunk - 1) / chunk; };
  auto len = [](int lo, int hi) { return hi - lo; };
  const Unit un = find_unit_quant<256>(offs, S, T, u, chunks, len);
  if (un.e >= 0) {
    const int t0 = un.lo + un.j * chunk;
    return TokenRange{un.e, t0, min(t0 + chunk, un.hi)};
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
};

template <int VPL, bool BF16, bool SIGMOID, bool GATE, bool BAL>
__global__ __launch_bounds__(256) void gate_kernel(GateFwd p) {
  __shared__ int s_cnt[BAL ? kGateMaxExperts : 1];
  __shared__ float s_sum[BAL ? 4 : 1][BAL ? 64 * VPL : 1];
  __shared__ int s_n[4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  TokenRange rg;
  if constexpr (BAL) {
    rg = gate_unit(p.offs, p.S, p.T, blockIdx.x, p.chunk);
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

  for (int t = rg.t0 + wave; t < rg.t1; t += 4) {
    const bool on = p.mask == nullptr || p.mask[t] != 0;   // wave-uniform
    const int64_t slot0 = (int64_t)t * p.topk;
    if (!on) {
      if constexpr (GATE) {
        if (lane < p.topk) {
          p.ids[slot0 + lane] = -1;
          p.weights[slot0 + lane] = 0.0f;
        }
      }
      continue;
    }
    float z[VPL], s[VPL];   // logits; scores up to the softmax's denominator
    float m = -kFltMax;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      const int e = lane + 64 * v;
      z[v] = e < p.E ? gate_logit<BF16>(p.logits, (int64_t)t * p.ld + e) : -INFINITY;
      m = fmaxf(m, z[v]);
    }
    if constexpr (!SIGMOID) m = gate_max(m);
    float total = 0.0f;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      s[v] = SIGMOID ? sigmoid_f32(z[v]) : __expf(z[v] - m);   // 0 for -inf
      total += s[v];
    }
    if constexpr (!SIGMOID || BAL) total = gate_sum(total);
    const float inv = total > 0.0f ? __fdiv_rn(1.0f, total) : 0.0f;

    int my_id = -1;   // lane j < topk: slot j
    if constexpr (GATE) {
      double key[VPL];
      if (p.bias == nullptr) {
#pragma unroll
        for (int v = 0; v < VPL; ++v) key[v] = gate_pack((double)z[v], lane + 64 * v);
      } else {
        double d[VPL], dt = 0.0;
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
          d[v] = SIGMOID ? 1.0 / (1.0 + exp(-(double)z[v])) : exp((double)z[v] - (double)m);
          dt += d[v];
        }
        if constexpr (!SIGMOID) dt = gate_sum(dt);
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
          const int e = lane + 64 * v;
          const double k = e < p.E ? (SIGMOID ? d[v] : d[v] / dt) + (double)p.bias[e] : 0.0;
          key[v] = z[v] > -INFINITY ? gate_pack(k, e) : -INFINITY;
        }
      }
      for (int j = 0; j < p.topk; ++j) {
        double best = -INFINITY;
#pragma unroll
        for (int v = 0; v < VPL; ++v) best = fmax(best, key[v]);
        best = gate_max(best);
        if (!(best > -INFINITY)) break;   // no eligible expert left (wave-uniform)
        if (lane == j) my_id = gate_index(best);
#pragma unroll
        for (int v = 0; v < VPL; ++v) key[v] = key[v] == best ? -INFINITY : key[v];
      }
      float w = 0.0f;
      if (my_id >= 0) {
        const float zj = gate_logit<BF16>(p.logits, (int64_t)t * p.ld + my_id);
        w = SIGMOID ? sigmoid_f32(zj) : __expf(zj - m);
      }
      if (p.renorm) {
        const float ws = gate_sum(w);
        w = ws > 0.0f ? __fdiv_rn(w, ws) : 0.0f;   // exactly 1 for a single choice
      } else if constexpr (!SIGMOID) {
        w *= inv;
      }
      if (lane < p.topk) {
        p.ids[slot0 + lane] = my_id;
        p.weights[slot0 + lane] = w * p.route_scale;
      }
    }
    if constexpr (BAL) {
      if (counted) {
        if constexpr (!GATE)
          if (lane < p.topk) my_id = p.ids[slot0 + lane];
        if (my_id >= 0 && my_id < p.E) atomicAdd(&s_cnt[my_id], 1);
        ++n;
#pragma unroll
        for (int v = 0; v < VPL; ++v) acc[v] += s[v] * inv;
      }
    }
  }
  if constexpr (BAL) {
#pragma unroll
    for (int v = 0; v < VPL; ++v) s_sum[wave][lane + 64 * v] = acc[v];
    if (lane == 0) s_n[wave] = n;
    __syncthreads();
    if (!counted) return;
    const int64_t at = (int64_t)blockIdx.x * p.E;
    for (int e = threadIdx.x; e < p.E; e += 256) {
      p.part_p[at + e] = (s_sum[0][e] + s_sum[1][e]) + (s_sum[2][e] + s_sum[3][e]);
      p.part_c[at + e] = s_cnt[e];
    }
    if (threadIdx.x == 0) p.part_n[blockIdx.x] = (s_n[0] + s_n[1]) + (s_n[2] + s_n[3]);
  }
}

// ---------------------------------------------------------------- the loss from the units' sums

struct GateLoss {
  int T, E, topk, chunk, S;
  float coef;
  const int32_t* offs;
  const float* part_p;
  const int32_t* part_c;
  const int32_t* part_n;
  double* seq_loss;    // [S]
  float* loss;         // written here with one sequence
  int32_t* counts;     // [S][E]
  float* dprob;        // [S][E]
};

// First unit and unit count of sequence s (workgroup-wide; the rule of find_unit).
template <int NT>
__device__ __forceinline__ void seq_units(const int32_t* __restrict__ offs, int S, int T, int s, int chunk, int& first,
                                          int& count) {
  if (offs == nullptr) {
    first = 0;
    count = (T + chunk - 1) / chunk;
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
    const int cnt = e < S ? (hi - lo + chunk - 1) / chunk : 0;
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

// One workgroup per sequence.
__global__ __launch_bounds__(256) void gate_loss_kernel(GateLoss p) {
  __shared__ double red[4];
  const int s = blockIdx.x;
  int first, count;
  seq_units<256>(p.offs, p.S, p.T, s, p.chunk, first, count);
  int n = 0;
  for (int u = 0; u < count; ++u) n += p.part_n[first + u];
  const double scale = (double)p.coef / p.S;
  double loss = 0.0;
  for (int e = threadIdx.x; e < p.E; e += 256) {
    double sum = 0.0;
    int c = 0;
#pragma unroll 4
    for (int u = 0; u < count; ++u) {
      sum += (double)p.part_p[(int64_t)(first + u) * p.E + e];
      c += p.part_c[(int64_t)(first + u) * p.E + e];
    }
    const double f = n > 0 ? (double)c * p.E / ((double)p.topk * n) : 0.0;
    loss += n > 0 ? f * sum / n : 0.0;
    p.counts[(int64_t)s * p.E + e] = c;
    p.dprob[(int64_t)s * p.E + e] = n > 0 ? (float)(scale * f / n) : 0.0f;
  }
  loss = gate_sum(loss);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = loss;
  __syncthreads();
  if (threadIdx.x == 0) {
    loss = scale * ((red[0] + red[1]) + (red[2] + red[3]));
    if (p.S == 1) *p.loss = (float)loss;
    else p.seq_loss[s] = loss;
  }
}

__global__ __launch_bounds__(64) void gate_loss_sum_kernel(const double* __restrict__ seq_loss, int S,
                                                           float* __restrict__ loss) {
  double t = 0.0;
  for (int s = threadIdx.x; s < S; s += 64) t += seq_loss[s];
  t = gate_sum(t);
  if (threadIdx.x == 0) *loss = (float)t;
}

// ---------------------------------------------------------------- backward
//
// With p the scores, ds the gradient reaching them:
//   softmax  dz = p (ds - sum p ds),    sigmoid  dz = ds p (1 - p).
// ds of a chosen expert: route_scale dw, or with renormalisation
// (route_scale dw - sum over slots of route_scale dw u) / (chosen scores' sum), u the
// normalised weights; plus the loss's dloss * dprob on the normalised scores.

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

template <int VPL, bool BF16, bool SIGMOID>
__global__ __launch_bounds__(256) void gate_bwd_kernel(GateBwd p) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  TokenRange rg;
  if (p.dprob != nullptr) {
    rg = gate_unit(p.offs, p.S, p.T, blockIdx.x, p.chunk);
  } else {
    const int64_t t0 = (int64_t)blockIdx.x * p.chunk;
    rg = TokenRange{-1, (int)min(t0, (int64_t)p.T), (int)min(t0 + p.chunk, (int64_t)p.T)};
  }
  const float dl = p.dloss != nullptr ? *p.dloss : 1.0f;
  for (int t = rg.t0 + wave; t < rg.t1; t += 4) {
    const bool on = p.mask == nullptr || p.mask[t] != 0;   // wave-uniform
    float z[VPL], s[VPL], ds[VPL];
    float m = -kFltMax;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      const int e = lane + 64 * v;
      z[v] = on && e < p.E ? gate_logit<BF16>(p.logits, (int64_t)t * p.ld + e) : -INFINITY;
      m = fmaxf(m, z[v]);
      ds[v] = 0.0f;
    }
    if (on) {
      if constexpr (!SIGMOID) m = gate_max(m);
      float total = 0.0f;
#pragma unroll
      for (int v = 0; v < VPL; ++v) {
        s[v] = SIGMOID ? sigmoid_f32(z[v]) : __expf(z[v] - m);
        total += s[v];
      }
      total = gate_sum(total);
      const float inv = total > 0.0f ? __fdiv_rn(1.0f, total) : 0.0f;
      if (rg.seq >= 0) {
        float dot = 0.0f;
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
          const int e = lane + 64 * v;
          ds[v] = e < p.E ? dl * p.dprob[(int64_t)rg.seq * p.E + e] : 0.0f;
          dot += ds[v] * s[v];
        }
        if constexpr (SIGMOID) {   // through the division by the scores' sum
          dot = gate_sum(dot) * inv;
#pragma unroll
          for (int v = 0; v < VPL; ++v) ds[v] = (ds[v] - dot) * inv;
        }
      }
      if (p.dweights != nullptr) {
        int id = -1;
        float dw = 0.0f, w = 0.0f;   // lane j: slot j
        if (lane < p.topk) id = p.ids[(int64_t)t * p.topk + lane];
        if (id < 0 || id >= p.E) id = -1;
        if (id >= 0) {
          dw = p.dweights[(int64_t)t * p.topk + lane] * p.route_scale;
          const float zj = gate_logit<BF16>(p.logits, (int64_t)t * p.ld + id);
          w = SIGMOID ? sigmoid_f32(zj) : __expf(zj - m);
        }
        if (p.renorm) {
          const float ws = gate_sum(w);
          const float u = ws > 0.0f ? __fdiv_rn(w, ws) : 0.0f;
          const float mean = gate_sum(dw * u);
          // the softmax's denominator cancels between the chosen scores and their sum
          dw = ws > 0.0f && id >= 0 ? (dw - mean) * __fdiv_rn(SIGMOID ? 1.0f : total, ws) : 0.0f;
        }
        for (int j = 0; j < p.topk; ++j) {
          const int ij = __shfl(id, j, 64);
          const float dj = __shfl(dw, j, 64);
#pragma unroll
          for (int v = 0; v < VPL; ++v) ds[v] += lane + 64 * v == ij ? dj : 0.0f;
        }
      }
      if constexpr (SIGMOID) {
#pragma unroll
        for (int v = 0; v < VPL; ++v) ds[v] *= s[v] * (1.0f - s[v]);
      } else {
        float dot = 0.0f;
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
          s[v] *= inv;
          dot += s[v] * ds[v];
        }
        dot = gate_sum(dot);
#pragma unroll
        for (int v = 0; v < VPL; ++v) ds[v] = s[v] * (ds[v] - dot);
      }
    }
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      const int e = lane + 64 * v;
      if (e < p.E) {
        if constexpr (BF16) static_cast<__bf16*>(p.dlogits)[(int64_t)t * p.E + e] = (__bf16)ds[v];
        else static_cast<float*>(p.dlogits)[(int64_t)t * p.E + e] = ds[v];
      }
    }
  }
}

// ---------------------------------------------------------------- launchers

template <typename F>
static hipError_t gate_dispatch(int E, bool bf16, bool sigmoid, F&& f) {
  auto types = [&](auto vpl) -> hipError_t {
    using T = std::true_type;
    using N = std::false_type;
    if (bf16) return sigmoid ? f(vpl, T{}, T{}) : f(vpl, T{}, N{});
    return sigmoid ? f(vpl, N{}, T{}) : f(vpl, N{}, N{});
  };
  if (E <= 64) return types(std::integral_constant<int, 1>{});
  if (E <= 128) return types(std::integral_constant<int, 2>{});
  if (E <= 256) return types(std::integral_constant<int, 4>{});
  if (E <= 512) return types(std::integral_constant<int, 8>{});
  return types(std::integral_constant<int, 16>{});
}

hipError_t launch_moe_gate(const GateArgs& a, hipStream_t st) {
  const bool gate = a.gate, bal = a.loss != nullptr;
  GateFwd p;
  p.logits = a.logits;
  p.ld = a.ld;
  p.T = (int)a.tokens;
  p.E = a.E;
  p.topk = a.topk;
  p.renorm = a.renorm;
  p.chunk = gate_chunk(a.tokens);
  p.S = a.S;
  p.bias = a.bias;
  p.mask = a.mask;
  p.route_scale = a.route_scale;
  p.ids = a.ids;
  p.weights = a.weights;
  p.offs = a.seq_offs;
  p.part_p = nullptr;
  p.part_c = nullptr;
  p.part_n = nullptr;
  const int64_t units = bal ? gate_units(a.tokens, a.S) : (a.tokens + p.chunk - 1) / p.chunk;
  double* seq_loss = nullptr;
  if (bal) {
    seq_loss = static_cast<double*>(a.workspace);
    p.part_p = reinterpret_cast<float*>(seq_loss + a.S);
    p.part_c = reinterpret_cast<int32_t*>(p.part_p + units * a.E);
    p.part_n = p.part_c + units * a.E;
  }
  if (a.tokens > 0) {
    const hipError_t e = gate_dispatch(a.E, a.bf16, a.sigmoid, [&](auto vpl, auto bf, auto sg) -> hipError_t {
      constexpr int V = decltype(vpl)::value;
      constexpr bool B = decltype(bf)::value, G = decltype(sg)::value;
      const dim3 grid((unsigned)units), block(256);
      if (gate && bal) hipLaunchKernelGGL((gate_kernel<V, B, G, true, true>), grid, block, 0, st, p);
      else if (gate) hipLaunchKernelGGL((gate_kernel<V, B, G, true, false>), grid, block, 0, st, p);
      else hipLaunchKernelGGL((gate_kernel<V, B, G, false, true>), grid, block, 0, st, p);
      return hipGetLastError();
    });
    if (e != hipSuccess) return e;
  }
  if (!bal) return hipSuccess;
  const GateLoss l{p.T,      p.E,      p.topk,   p.chunk,  a.S,    a.coef,   a.seq_offs,
                   p.part_p, p.part_c, p.part_n, seq_loss, a.loss, a.counts, a.dprob};
  hipLaunchKernelGGL(gate_loss_kernel, dim3((unsigned)a.S), dim3(256), 0, st, l);
  if (a.S > 1) hipLaunchKernelGGL(gate_loss_sum_kernel, dim3(1), dim3(64), 0, st, seq_loss, a.S, a.loss);
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
  p.chunk = gate_chunk(a.tokens);
  p.S = a.S;
  p.mask = a.mask;
  p.route_scale = a.route_scale;
  p.ids = a.ids;
  p.dweights = a.dweights;
  p.offs = a.seq_offs;
  p.dprob = a.dprob;
  p.dloss = a.dloss;
  p.dlogits = a.dlogits;
  const int64_t units = a.dprob != nullptr ? gate_units(a.tokens, a.S) : (a.tokens + p.chunk - 1) / p.chunk;
  return gate_dispatch(a.E, a.bf16, a.sigmoid, [&](auto vpl, auto bf, auto sg) -> hipError_t {
    constexpr int V = decltype(vpl)::value;
    hipLaunchKernelGGL((gate_bwd_kernel<V, decltype(bf)::value, decltype(sg)::value>), dim3((unsigned)units), dim3(256),
                       0, st, p);
    return hipGetLastError();
  });
}

}  // namespace fp8moe
