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

}  // namespace moe
