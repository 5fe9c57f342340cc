// Gradients of the top-k weighted reduce.
//
//   d_y_perm[inv_perm[t, j], :] = topk_w[t, j] * d_out[t, :]
//   d_topk_w[t, j]              = sum_h d_out[t, h] * y_perm[inv_perm[t, j], h]
//
// HBM-bound: d_out and the routed rows of y_perm are read once, the routed rows
// of d_y_perm written once.  A block owns one token; each thread holds float4
// columns of d_out and one partial dot product per slot, which the block sums
// in a fixed order (no atomics).
#include "operators.h"

namespace moe {
namespace {

constexpr int kThreads = 256;

// KS >= k slots (unrolled, guarded by k).
template <int KS>
__global__ __launch_bounds__(kThreads) void combine_backward_kernel(
    const floatx4* __restrict__ d_out, const floatx4* __restrict__ y_perm, const int32_t* __restrict__ inv_perm,
    const float* __restrict__ topk_w, int k, int H4, int64_t R_cap, floatx4* __restrict__ d_y,
    float* __restrict__ d_w) {
  __shared__ float s_part[kThreads / kWave][KS];
  const int64_t t = blockIdx.x;
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  int row[KS];
  float w[KS], dot[KS];
#pragma unroll
  for (int j = 0; j < KS; ++j) {
    const int p = j < k ? inv_perm[t * k + j] : -1;
    row[j] = (p >= 0 && p < R_cap) ? p : -1;
    w[j] = j < k ? topk_w[t * k + j] : 0.f;
    dot[j] = 0.f;
  }
  for (int c = threadIdx.x; c < H4; c += kThreads) {
    const floatx4 g = __builtin_nontemporal_load(d_out + t * H4 + c);
    floatx4 y[KS];
#pragma unroll
    for (int j = 0; j < KS; ++j)
      if (row[j] >= 0) y[j] = __builtin_nontemporal_load(y_perm + (int64_t)row[j] * H4 + c);
#pragma unroll
    for (int j = 0; j < KS; ++j)
      if (row[j] >= 0) {
        __builtin_nontemporal_store(w[j] * g, d_y + (int64_t)row[j] * H4 + c);
        const floatx4 p = g * y[j];
        dot[j] += (p[0] + p[1]) + (p[2] + p[3]);
      }
  }
#pragma unroll
  for (int j = 0; j < KS; ++j) {
    float v = dot[j];
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off);
    if (lane == 0) s_part[wv][j] = v;
  }
  __syncthreads();
  if ((int)threadIdx.x < k)
    d_w[t * k + threadIdx.x] = (s_part[0][threadIdx.x] + s_part[1][threadIdx.x]) +
                               (s_part[2][threadIdx.x] + s_part[3][threadIdx.x]);
}

}  // namespace

hipError_t launch_combine_backward(const float* d_out, const float* y_perm, const int32_t* inv_perm,
                                   const float* topk_w, int64_t T, int k, int H, int64_t R_cap, float* d_y_perm,
                                   float* d_topk_w, hipStream_t s) {
  const int H4 = H / 4;
  const floatx4* g = reinterpret_cast<const floatx4*>(d_out);
  const floatx4* y = reinterpret_cast<const floatx4*>(y_perm);
  floatx4* d_y = reinterpret_cast<floatx4*>(d_y_perm);
#define MOE_COMBINE_BWD(KS_)                                                                                 \
  hipLaunchKernelGGL(combine_backward_kernel<KS_>, dim3((unsigned)T), dim3(kThreads), 0, s, g, y, inv_perm, \
                     topk_w, k, H4, R_cap, d_y, d_topk_w)
  if (k <= 1) MOE_COMBINE_BWD(1);
  else if (k <= 2) MOE_COMBINE_BWD(2);
  else if (k <= 4) MOE_COMBINE_BWD(4);
  else if (k <= 8) MOE_COMBINE_BWD(8);
  else if (k <= 16) MOE_COMBINE_BWD(16);
  else MOE_COMBINE_BWD(32);
#undef MOE_COMBINE_BWD
  return hipGetLastError();
}

}  // namespace moe
