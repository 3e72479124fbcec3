// Sums and maxima over aligned groups of 4, 16 or 64 lanes on the VALU (no LDS
// wait): quad permutations for 4 lanes, rotations of a 16-lane row by 8, 4, 2, 1
// (after a rotation by 2^k the value has period 2^k along the row), gfx950's row
// swaps across rows.  Every lane of the group ends with the same bits: each step
// combines two values that both partners hold, and the operations commute.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp8moe {

// (bound_ctrl set: no lane reads outside its row here, and the compiler then folds the exchange into the operation.)
template <int CTL>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTL, 0xF, 0xF, true);
}
template <int CTL>
__device__ __forceinline__ float dpp_f32(float v) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTL, 0xF, 0xF, true));
}
template <int CTL>
__device__ __forceinline__ double dpp_f64(double v) {
  const int64_t b = __double_as_longlong(v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_mov_dpp((int)b, CTL, 0xF, 0xF, true);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_mov_dpp((int)(b >> 32), CTL, 0xF, 0xF, true);
  return __longlong_as_double((int64_t)(((uint64_t)hi << 32) | lo));
}

template <int N, typename Op>
__device__ __forceinline__ float group_reduce_f32(float v, Op op) {
  static_assert(N == 4 || N == 16 || N == 64, "group size");
  if constexpr (N == 4) {
    v = op(v, dpp_f32<0xB1>(v));   // quad_perm [1,0,3,2]
    return op(v, dpp_f32<0x4E>(v));   // quad_perm [2,3,0,1]
  } else {
    v = op(v, dpp_f32<0x128>(v));   // row_ror:8
    v = op(v, dpp_f32<0x124>(v));
    v = op(v, dpp_f32<0x122>(v));
    v = op(v, dpp_f32<0x121>(v));
    if constexpr (N == 64) {
      const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
      v = op(__uint_as_float(a[0]), __uint_as_float(a[1]));
      const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
      v = op(__uint_as_float(b[0]), __uint_as_float(b[1]));
    }
    return v;
  }
}
template <int N>
__device__ __forceinline__ uint32_t group_most_u32(uint32_t v) {
  static_assert(N == 4 || N == 16 || N == 64, "group size");
  if constexpr (N == 4) {
    v = max(v, dpp_u32<0xB1>(v));
    return max(v, dpp_u32<0x4E>(v));
  } else {
    v = max(v, dpp_u32<0x128>(v));
    v = max(v, dpp_u32<0x124>(v));
    v = max(v, dpp_u32<0x122>(v));
    v = max(v, dpp_u32<0x121>(v));
    if constexpr (N == 64) {
      const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
      v = max(a[0], a[1]);
      const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
      v = max(b[0], b[1]);
    }
    return v;
  }
}
template <int N>
__device__ __forceinline__ float group_sum_f32(float v) {
  return group_reduce_f32<N>(v, [](float a, float b) { return a + b; });
}
template <int N>
__device__ __forceinline__ float group_max_f32(float v) {
  return group_reduce_f32<N>(v, [](float a, float b) { return fmaxf(a, b); });
}

template <int N, typename Op>
__device__ __forceinline__ double group_reduce_f64(double v, Op op) {
  static_assert(N == 4 || N == 16 || N == 64, "group size");
  if constexpr (N == 4) {
    v = op(v, dpp_f64<0xB1>(v));
    return op(v, dpp_f64<0x4E>(v));
  } else {
    v = op(v, dpp_f64<0x128>(v));
    v = op(v, dpp_f64<0x124>(v));
    v = op(v, dpp_f64<0x122>(v));
    v = op(v, dpp_f64<0x121>(v));
    if constexpr (N == 64) {
      auto swap = [&](auto swap32) {
        const int64_t b = __double_as_longlong(v);
        const uint32_t l = (uint32_t)b, h = (uint32_t)(b >> 32);
        uint32_t l0, l1, h0, h1;
        if constexpr (decltype(swap32)::value) {
          const auto x = __builtin_amdgcn_permlane32_swap(l, l, false, false);
          const auto y = __builtin_amdgcn_permlane32_swap(h, h, false, false);
          l0 = x[0], l1 = x[1], h0 = y[0], h1 = y[1];
        } else {
          const auto x = __builtin_amdgcn_permlane16_swap(l, l, false, false);
          const auto y = __builtin_amdgcn_permlane16_swap(h, h, false, false);
          l0 = x[0], l1 = x[1], h0 = y[0], h1 = y[1];
        }
        v = op(__longlong_as_double((int64_t)(((uint64_t)h0 << 32) | l0)),
               __longlong_as_double((int64_t)(((uint64_t)h1 << 32) | l1)));
      };
      swap(std::false_type{});
      swap(std::true_type{});
    }
    return v;
  }
}
template <int N>
__device__ __forceinline__ double group_sum_f64(double v) {
  return group_reduce_f64<N>(v, [](double a, double b) { return a + b; });
}
template <int N>
__device__ __forceinline__ double group_max_f64(double v) {
  return group_reduce_f64<N>(v, [](double a, double b) { return fmax(a, b); });
}

}  // namespace fp8moe
