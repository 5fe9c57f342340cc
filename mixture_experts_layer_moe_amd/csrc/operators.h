// Internal launchers of the operators beside the four-call path (grouped
// routing, gradients, dense projection); called by moe_api.hip after argument
// validation.  All return hipGetLastError() after launching.
#pragma once

#include "common.h"

namespace moe {

struct RouteArgs {
  const float* logits;
  const float* bias;  // may be null
  int64_t T;
  int E, k;
  bool sigmoid, renormalize;
  int n_group, topk_group, group_top;
  float scale;
  int32_t* idx;
  float* w;
};
hipError_t launch_route_grouped(const RouteArgs& a, hipStream_t s);

struct RouteBwdArgs {
  const float* logits;
  const float* bias;  // may be null
  const int32_t* idx;
  const float* d_w;
  int64_t T;
  int E, k;
  bool sigmoid, renormalize;
  float scale;
  float* d_logits;
};
hipError_t launch_route_grouped_backward(const RouteBwdArgs& a, hipStream_t s);

hipError_t launch_combine_backward(const float* d_out, const float* y_perm, const int32_t* inv_perm,
                                   const float* topk_w, int64_t T, int k, int H, int64_t R_cap, float* d_y_perm,
                                   float* d_topk_w, hipStream_t s);

// Activations of the dense projection (moe_act and the MOE_ACT_* values of the header).
enum LinearAct { ACT_GELU = 0, ACT_SWIGLU = 1, ACT_NONE = 2, ACT_SILU = 3 };

struct LinearArgs {
  const uint16_t *x, *w, *w_up;  // w_up: SwiGLU only
  const float *bias, *bias_up;
  const void* residual;
  int64_t M;
  int N, K, act;
  bool out_f32;
  uint16_t *z, *z_up;
  void* out;
  void* ws;  // may be null: the reduction is not split
};
size_t linear_ws_bytes(int64_t M, int N, int K, int act);
hipError_t launch_linear(const LinearArgs& a, hipStream_t s);

struct LinearBwdArgs {
  const void* d_out;
  const uint16_t *x, *w, *w_up, *z, *z_up;
  int64_t M;
  int N, K, act;
  bool out_f32;
  uint16_t *d_x, *d_w, *d_w_up;
  float *d_bias, *d_bias_up;
  void* ws;
};
size_t linear_backward_ws_bytes(int64_t M, int N, int K, int act);
hipError_t launch_linear_backward(const LinearBwdArgs& a, hipStream_t s);

// MXFP4 (codes of two values a byte, a scale byte per 32 values).
hipError_t launch_mxfp4_quantize(const void* x, bool f32, int64_t blocks, uint8_t* codes, uint8_t* scales, hipStream_t s);
hipError_t launch_mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t blocks, bool f32, void* out,
                                   hipStream_t s);

struct Mx {
  const uint8_t *q, *s;  // codes, scales
};
struct MxLinearArgs {
  Mx x, w, w_up;  // w_up: SwiGLU only
  const float *bias, *bias_up;
  const void* residual;
  int64_t M;  // dense: rows; grouped: rows of x
  int N, K, act;
  bool out_f32;
  void* out;
  // Grouped: row tiles of the permutation (counts null: dense).
  const int32_t *counts, *offsets, *tiles, *num_tiles, *row_src;  // row_src null: x's rows are the permuted ones
  int topk, tile_m, E_loc;
  int64_t tiles_cap, R_cap;
};
hipError_t launch_linear_mxfp4(const MxLinearArgs& a, hipStream_t s);
hipError_t launch_grouped_linear_mxfp4(const MxLinearArgs& a, hipStream_t s);

// A whole layer for at most kFewTokens tokens.
constexpr int kFewTokens = 64;
struct FewArgs {
  const uint16_t* x;
  const float* logits;  // null: topk_idx and topk_w are given
  int T, E, k, expert_begin, E_loc, H, F;
  bool renormalize;
  const void *w0, *w0_up, *w1;           // bf16, or MXFP4 codes; w0_up null: GELU, else SwiGLU
  const uint8_t *s0, *s0_up, *s1;        // MXFP4 scales, or null
  int32_t* topk_idx;
  float* topk_w;
  float* out;
  void* ws;
};
size_t few_tokens_ws_bytes(int T, int k, int F);
hipError_t launch_few_tokens(const FewArgs& a, hipStream_t s);

}  // namespace moe
