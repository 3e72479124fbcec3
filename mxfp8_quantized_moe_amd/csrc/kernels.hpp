// Internal launchers: one per operation, called by the C ABI after validation.
// Each enqueues kernels on `st` and returns hipGetLastError().
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

namespace fp8moe {

// Compute units of the current device (queried once per device).
int device_cu_count();

hipError_t launch_quantize_rowwise(const uint16_t* x, int64_t rows, int64_t cols, int64_t ld_x, int codec,
                                   uint8_t* q, float* scale, hipStream_t st);

hipError_t launch_moe_permute_colwise(const uint16_t* x, int64_t tokens, int64_t cols, int topk, const int32_t* src,
                                      const float* weights, int64_t rows, const int32_t* offs, int32_t n_groups,
                                      int codec, uint8_t* q_t, int64_t ld_q, float* scale, hipStream_t st);
hipError_t launch_quantize_colwise(const uint16_t* x, int64_t batch, int64_t rows, int64_t cols,
                                   const int32_t* offs, int32_t n_groups, int codec, uint8_t* q_t,
                                   int64_t ld_q, float* scale, hipStream_t st);

hipError_t launch_quantize_mx(const uint16_t* x, int64_t batch, int64_t rows, int64_t cols, int axis,
                              const int32_t* offs, int32_t n_groups, int rule, int scale_layout, uint8_t* q,
                              uint8_t* sc, int64_t rows_pad, int32_t* offs_pad_out, hipStream_t st);

hipError_t launch_quantize_mx_dual(const uint16_t* x, int64_t batch, int64_t rows, int64_t cols,
                                   const int32_t* offs, int32_t n_groups, int rule, int scale_layout, uint8_t* q,
                                   uint8_t* sc, uint8_t* q_t, uint8_t* sc_t, int64_t rows_pad,
                                   int32_t* offs_pad_out, hipStream_t st);

// SwiGLU (da2 null) or its backward (da2 given) computed on the fly and quantized into both MX forms.
hipError_t launch_moe_permute_mx_dual(const uint16_t* x, int64_t tokens, int64_t cols, int topk, const int32_t* src,
                                     const float* weights, int64_t rows, const int32_t* offs, int32_t n_groups,
                                     int rule, int scale_layout, uint16_t* xg, uint8_t* q, uint8_t* sc, uint8_t* q_t,
                                     uint8_t* sc_t, int64_t rows_pad, int32_t* offs_pad_out, hipStream_t st);
hipError_t launch_swiglu_mx_dual(const uint16_t* h1, const uint16_t* da2, bool bwd, int64_t rows, int64_t F,
                                 int64_t ld_h1, const int32_t* offs, int32_t n_groups, int rule, int scale_layout, uint16_t* out,
                                 uint8_t* q, uint8_t* sc, uint8_t* q_t, uint8_t* sc_t, int64_t rows_pad,
                                 int32_t* offs_pad_out, hipStream_t st);

struct GemmArgs {
  int mode, a_fmt, b_fmt, scale_kind, out_dtype;
  const void* a;
  const void* b;
  const void* sa;
  const void* sb;
  const int32_t* offs;
  int n_groups;
  int64_t M, N, K;
  void* out;
};

hipError_t launch_grouped_mm(const GemmArgs& g, hipStream_t st);
// Integer operands with few rows a group.
bool i8_rows_wanted(const GemmArgs& g);
hipError_t launch_i8_rows(const GemmArgs& g, hipStream_t st);

// Poll budget of the single-pass colwise exchange (negative: the default); returns the previous one.
int set_colwise_poll_budget(int polls);
// Chunk height of the single-pass colwise quantizer (128 or 512: forced; else per call); returns the previous one.
int set_colwise_chunk_rows(int rows);

hipError_t launch_encode_f32(const float* y, int64_t n, int codec, uint8_t* q, hipStream_t st);
hipError_t launch_quantize_blockwise(const uint16_t* x, int64_t batch, int64_t rows, int64_t cols, int block_rows,
                                     int codec, uint8_t* q, float* scale, hipStream_t st);
hipError_t launch_grouped_mm_blockwise(const uint8_t* a, const float* sa, const uint8_t* b, const float* sb,
                                       const int32_t* offs, int n_groups, int64_t M, int64_t N, int64_t K, void* out,
                                       int out_dtype, hipStream_t st);
hipError_t launch_quantize_blockwise_tokens(const uint16_t* x, int64_t M, int64_t C, const int32_t* offs, int n_groups,
                                            int codec, uint8_t* q_t, int64_t ld_q, float* scale, hipStream_t st);
hipError_t launch_grouped_mm_blockwise_k(const uint8_t* a_t, const float* sa, const uint8_t* b_t, const float* sb,
                                         const int32_t* offs, int n_groups, int64_t M, int64_t ld, int64_t N,
                                         int64_t K, void* out, int out_dtype, hipStream_t st);
hipError_t launch_quantize_tensorwise(const uint16_t* x, int64_t batch, int64_t rows, int64_t cols, int codec,
                                      uint8_t* q, uint8_t* q_t, int64_t ld_q, float* scale, int64_t n_scale,
                                      uint32_t* part, hipStream_t st);
hipError_t launch_moe_route(const int32_t* ids, int64_t S, int E, int pad, int32_t* counts, int32_t* offs,
                            int32_t* dest, int32_t* src, int64_t rows_bound, int32_t* workspace, hipStream_t st);
hipError_t launch_moe_route_noalloc(const int32_t* ids, int64_t S, int E, int pad, int32_t* counts, int32_t* offs,
                                    int32_t* dest, int32_t* src, int64_t rows_bound, hipStream_t st);
hipError_t launch_moe_permute(const uint16_t* x, int64_t tokens, int64_t cols, int topk, const int32_t* src,
                              int64_t rows_out, uint16_t* xg, hipStream_t st);
hipError_t launch_moe_permute_quantized(const uint8_t* q, const float* scale, int64_t tokens, int64_t cols, int topk,
                                        const int32_t* src, int64_t rows_out, int codec, uint8_t* qg,
                                        float* scale_g, hipStream_t st);
hipError_t launch_moe_combine(const uint16_t* yg, int64_t rows_in, const int32_t* dest, const float* w,
                              int64_t tokens, int topk, int64_t cols, uint16_t* y, hipStream_t st);
hipError_t launch_moe_permute_rowwise(const uint16_t* x, int64_t tokens, int64_t cols, int topk, const int32_t* src,
                                      int64_t rows_out, int codec, uint16_t* xg, uint8_t* qg, float* scale_g,
                                      hipStream_t st);
hipError_t launch_moe_combine_backward(const uint16_t* dy, const uint16_t* yg, int64_t rows, const int32_t* dest,
                                       const int32_t* src, const float* w, int64_t tokens, int topk, int64_t cols,
                                       int codec, uint16_t* dyg, uint8_t* q, float* scale, float* dw,
                                       hipStream_t st);
hipError_t launch_swiglu_quantize_rowwise(const uint16_t* h1, int64_t rows, int64_t F, int64_t ld_h1, int codec,
                                          uint16_t* a2, uint8_t* q, float* scale, hipStream_t st);
hipError_t launch_swiglu_backward_quantize_rowwise(const uint16_t* da2, const uint16_t* h1, int64_t rows, int64_t F,
                                                   int64_t ld_h1, int codec, uint16_t* dh1, uint8_t* q, float* scale,
                                                   hipStream_t st);


// RMS norm with a quantized output.  fmt 0, 1: rowwise codes of that codec; 2, 3: MX under the floor, ceil
// rule; 4: no codes.
struct NormArgs {
  const uint16_t* x;
  const uint16_t* res;
  const void* gamma;
  bool gamma_bf16;
  int64_t rows, cols, ld_x, ld_r;
  float eps;
  int fmt, layout;
  uint16_t* sum;
  uint16_t* h;
  uint8_t* q;
  float* scale;
  uint8_t* sc;
  float* rstd;
};
hipError_t launch_rmsnorm_quantize(const NormArgs& a, hipStream_t st);
hipError_t launch_rmsnorm_backward(const uint16_t* dh, const uint16_t* s, const float* rstd, const void* gamma,
                                   bool gamma_bf16, const uint16_t* dsum, int64_t rows, int64_t cols, uint16_t* dx,
                                   float* dgamma, float* workspace, hipStream_t st);

// Router gate and balance loss (either or both): gate writes ids and weights, loss non-null asks for the loss.
struct GateArgs {
  const void* logits;
  bool bf16, sigmoid, gate;
  int64_t tokens, ld;
  int E, topk;
  const float* bias;
  const uint8_t* mask;
  int renorm;
  float route_scale;
  int32_t* ids;
  float* weights;
  const int32_t* seq_offs;
  int S;
  float coef;
  float* loss;
  int32_t* counts;
  float* dprob;
  void* workspace;
};
hipError_t launch_moe_gate(const GateArgs& a, hipStream_t st);
struct GateBwdArgs {
  const void* logits;
  bool bf16, sigmoid;
  int64_t tokens, ld;
  int E, topk;
  const uint8_t* mask;
  int renorm;
  float route_scale;
  const int32_t* ids;
  const float* dweights;
  const int32_t* seq_offs;
  int S;
  const float* dprob;
  const float* dloss;
  void* dlogits;
};
hipError_t launch_moe_gate_backward(const GateBwdArgs& a, hipStream_t st);

// The expert block for a few tokens.  fmt 0: e4m3fn with fp32 row scales, 1: int8 with fp32 row scales, 2, 3: MXFP8
// with row-major, K4 scales.
struct FewArgs {
  const uint16_t* x;
  int64_t ld_x;
  const int32_t* ids;
  const float* weights;
  int64_t tokens;
  int topk, n_experts;
  int64_t K, F;
  const uint8_t* w1;
  const uint8_t* w2;
  const void* s1;
  const void* s2;
  int fmt;
  void* workspace;
  uint16_t* y;
};
hipError_t launch_moe_few_tokens(const FewArgs& a, hipStream_t st);

// SwiGLU with its input kept in MXFP8, and what reads it (da2 null: SwiGLU, else its backward).
hipError_t launch_swiglu_save(const uint16_t* h1, int64_t rows, int64_t F, int64_t ld_h1, int codec, int rule,
                              uint16_t* a2, uint8_t* q, float* scale, uint8_t* hq, uint8_t* hs, hipStream_t st);
hipError_t launch_swiglu_saved_backward(const uint16_t* da2, const uint8_t* hq, const uint8_t* hs, int64_t rows, int64_t F,
                                        int codec, uint16_t* dh1, uint8_t* q, float* scale, uint16_t* a2, hipStream_t st);
hipError_t launch_swiglu_mx_dual_saved(const uint8_t* hq, const uint8_t* hs, const uint16_t* da2, bool bwd, int64_t rows,
                                       int64_t F, const int32_t* offs, int32_t n_groups, int rule, int scale_layout, uint16_t* out,
                                       uint8_t* q, uint8_t* sc, uint8_t* q_t, uint8_t* sc_t, int64_t rows_pad,
                                       int32_t* offs_pad_out, hipStream_t st);

}  // namespace fp8moe
