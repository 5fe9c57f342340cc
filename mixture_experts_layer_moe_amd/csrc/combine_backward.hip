// Gradients of the top-k weighted reduce.
//
//   d_y_perm[inv_perm[t, j], :] = topk_w[t, j] * d_out[t, :]
//   d_topk_w[t, j]              = sum_h d_out[t, h] * y_perm[inv_perm[t, j], h]
//
// HBM-bound: d_out and the routed rows of y_perm are read once, the routed rows
// of d_y_perm written once.  A block owns one token and holds V float4 columns
// of d_out a thread; it takes the token's local slots one by one, the next
// slot's row in flight while one is used, and adds the block's partial dot
// products in a fixed order (no atomics).  4096 tokens of 4096 columns, two local slots each: 336 MB in 63 us (5.3
// TB/s; a copy of 1 GiB reaches 5.1); 5003 tokens, 8 slots of which about one is local: 247 MB in 47 us (all slots'
// rows at once, the absent ones masked, took 58).  Rows under 1024 columns leave threads without work: 16384 tokens of
// 256 columns 84 MB in 31 us.
#include "operators.h"

namespace moe {
namespace {

constexpr int kThreads = 256;

// Sum over the wavefront, in every lane: quad swaps and mirrors inside a row of 16 lanes, then the four rows.
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  const int x = __builtin_bit_cast(int, v);
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(x, x, CTRL, 0xF, 0xF, false));
}
__device__ __forceinline__ float of_lane(float v, int l) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), l));
}
__device__ __forceinline__ float wave_sum(float v) {
  v += dpp<0xB1>(v);
  v += dpp<0x4E>(v);
  v += dpp<0x141>(v);
  v += dpp<0x140>(v);
  return (of_lane(v, 0) + of_lane(v, 16)) + (of_lane(v, 32) + of_lane(v, 48));
}

// V: float4 columns per thread and span of a row (a block covers up to 4096 columns at once).
template <int V>
__global__ __launch_bounds__(kThreads) void combine_backward_kernel(
    const floatx4* __restrict__ d_out, const floatx4* __restrict__ y_perm, const int32_t* __restrict__ inv_perm,
    const float* __restrict__ topk_w, int k, int H4, int64_t R_cap, floatx4* __restrict__ d_y,
    float* __restrict__ d_w) {
  __shared__ float s_part[kThreads / kWave][32];
  const int64_t t = blockIdx.x;
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  // The token's next local slot after j (k: none) and its row; block-uniform.
  auto next = [&](int& j, int64_t& row) {
    for (++j; j < k; ++j) {
      row = inv_perm[t * k + j];
      if (row >= 0 && row < R_cap) break;
    }
  };
  if (lane < 32) s_part[wv][lane] = 0.f;
  for (int c0 = threadIdx.x; c0 - (int)threadIdx.x < H4; c0 += kThreads * V) {
    floatx4 g[V], y[2][V];
    auto load = [&](floatx4 (&x)[V], const floatx4* p) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = c0 + v * kThreads;
        x[v] = c < H4 ? __builtin_nontemporal_load(p + c) : floatx4{0.f, 0.f, 0.f, 0.f};
      }
    };
    load(g, d_out + t * H4);
    int j = -1, jn;
    int64_t row = 0, rn = 0;
    next(j, row);
    if (j < k) load(y[0], y_perm + row * H4);
    while (j < k) {
      jn = j;
      next(jn, rn);
      if (jn < k) load(y[1], y_perm + rn * H4);
      const float w = topk_w[t * k + j];
      float dot = 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = c0 + v * kThreads;
        if (c < H4) __builtin_nontemporal_store(w * g[v], d_y + row * H4 + c);
        const floatx4 p = g[v] * y[0][v];
        dot += (p[0] + p[1]) + (p[2] + p[3]);
      }
      dot = wave_sum(dot);
      if (lane == 0) s_part[wv][j] += dot;
#pragma unroll
      for (int v = 0; v < V; ++v) y[0][v] = y[1][v];
      j = jn;
      row = rn;
    }
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
  constexpr int64_t kMaxTokens = 1 << 23;  // per launch (a grid holds fewer than 2^32 threads)
#define MOE_COMBINE_BWD(V_)                                                                                       \
  hipLaunchKernelGGL(combine_backward_kernel<V_>, dim3(n), dim3(kThreads), 0, s, g + t * H4, y, inv_perm + t * k, \
                     topk_w + t * k, k, H4, R_cap, d_y, d_topk_w + t * k)
  for (int64_t t = 0; t < T; t += kMaxTokens) {
    const unsigned n = (unsigned)(T - t < kMaxTokens ? T - t : kMaxTokens);
    // Columns per thread: a row in one span if it has 4096 columns or fewer.
    if (H4 > 2 * kThreads) MOE_COMBINE_BWD(4);
    else if (H4 > kThreads) MOE_COMBINE_BWD(2);
    else MOE_COMBINE_BWD(1);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
#undef MOE_COMBINE_BWD
  return hipSuccess;
}

}  // namespace moe
