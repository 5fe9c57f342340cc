// Routing with softmax or sigmoid scores, a bias for balance, expert groups
// and a scale, and the gradient of its gate weights.
//
//   s_e   = 1 / (1 + e^-l_e)   or   e^(l_e - m) / sum_f e^(l_f - m),  m the row's largest logit
//   key_e = s_e + bias_e; a group's key is the sum of its group_top largest; the topk_group best groups stay
//   the k largest keys among them, ties lowest id first;  w_j = scale * s_j (/ sum_i s_i)
//
// The choice has to be the one that exact arithmetic makes.  Both scores grow
// strictly with the logit, so without a bias experts (and groups ranked by
// their best expert) are compared by their logits, exactly.  Keys with a bias
// and sums of two scores are 64-bit: two of them that differ by less than an
// fp32 rounding are met every few thousand tokens.
//
// One wavefront per token; lane l holds experts l, l + 64, ...
#include "operators.h"

#include <float.h>

namespace moe {
namespace {

__device__ __forceinline__ float wave_max_f(float v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v = fmaxf(v, __shfl_xor(v, off));
  return v;
}
__device__ __forceinline__ float wave_sum_f(float v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off);
  return v;
}
__device__ __forceinline__ double wave_max_d(double v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v = fmax(v, __shfl_xor(v, off));
  return v;
}
__device__ __forceinline__ double wave_sum_d(double v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off);
  return v;
}
__device__ __forceinline__ double sigmoid_d(double x) { return 1.0 / (1.0 + exp(-x)); }
__device__ __forceinline__ int wave_min_i(int v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v = min(v, __shfl_xor(v, off));
  return v;
}

// e / Eg for e < 1024: magic = ceil(2^22 / Eg), exact because e * Eg < 2^22.
__device__ __forceinline__ int group_of(int e, uint32_t magic) { return (int)(((uint32_t)e * magic) >> 22); }

// A row's gate weights.  Lane j < k holds slot j's id (-1: empty) and logit; m is the row's largest available
// logit and z the sum of e^(l - m) over the available experts (used by the plain softmax only).
// Renormalised, both scores are scaled by a common factor that keeps the largest at least 1/2 before the sum:
// softmax by e^-(largest chosen logit), sigmoid(l) = e^min(l, 0) / (1 + e^-|l|) by e^-min(largest chosen logit, 0).
__device__ __forceinline__ float gate_weight(int lane, int k, int id, float l, float m, float z, bool sigmoid,
                                             bool renormalize, float scale) {
  const bool has = lane < k && id >= 0;
  float s = 0.f;
  if (renormalize) {
    float top = wave_max_f(has ? l : -FLT_MAX);
    if (sigmoid) top = fminf(top, 0.f);
    if (has) s = sigmoid ? expf(fminf(l, 0.f) - top) / (1.f + expf(-fabsf(l))) : expf(l - top);
    const float sum = wave_sum_f(s);
    return has ? scale * (s / sum) : 0.f;
  }
  if (has) s = sigmoid ? 1.f / (1.f + expf(-l)) : expf(l - m) / z;
  return scale * s;
}

constexpr int kTokens = 4;  // wavefronts (tokens) per block

// Dynamic LDS: per wavefront E keys (n_group > 1 only).
template <int PL>
__global__ __launch_bounds__(kTokens* kWave) void route_grouped_kernel(RouteArgs a, uint32_t magic) {
  extern __shared__ double s_key[];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int64_t t = (int64_t)blockIdx.x * kTokens + wv;
  const bool live = t < a.T;  // wave-uniform
  const int E = a.E;
  float l[PL];
  double key[PL];
  bool ok[PL];
  float m = -FLT_MAX;
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    const int e = lane + i * kWave;
    const float v = (live && e < E) ? a.logits[t * E + e] : -INFINITY;
    const float b = (a.bias && e < E) ? a.bias[e] : 0.f;
    ok[i] = v > -INFINITY && b > -INFINITY;  // false for NaN
    l[i] = fminf(v, FLT_MAX);
    if (ok[i]) m = fmaxf(m, l[i]);
  }
  m = wave_max_f(m);
  float z = 1.f;
  if (!a.sigmoid && !a.renormalize) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < PL; ++i) s += ok[i] ? expf(l[i] - m) : 0.f;
    z = wave_sum_f(s);
  }
  if (!a.bias) {
#pragma unroll
    for (int i = 0; i < PL; ++i) key[i] = l[i];
  } else {
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      key[i] = ok[i] ? (a.sigmoid ? sigmoid_d(l[i]) : exp((double)l[i] - (double)m)) : 0.0;
      s += key[i];
    }
    if (!a.sigmoid) {
      const double zz = wave_sum_d(s);
#pragma unroll
      for (int i = 0; i < PL; ++i) key[i] /= zz;
    }
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      const int e = lane + i * kWave;
      if (ok[i]) key[i] += (double)fminf(a.bias[e], FLT_MAX);
    }
  }
#pragma unroll
  for (int i = 0; i < PL; ++i)
    if (!ok[i]) key[i] = -INFINITY;

  if (a.n_group > 1 && a.topk_group < a.n_group) {
    double* sk = s_key + wv * E;
    const int Eg = E / a.n_group;
#pragma unroll
    for (int i = 0; i < PL; ++i)
      if (lane + i * kWave < E) sk[lane + i * kWave] = key[i];
    __syncthreads();
    double g = -INFINITY, g2 = -INFINITY;
    if (lane < a.n_group)
      for (int q = 0; q < Eg; ++q) {
        const double v = sk[lane * Eg + q];
        if (v > g) {
          g2 = g;
          g = v;
        } else if (v > g2) {
          g2 = v;
        }
      }
    if (a.group_top == 2 && g > -INFINITY) {
      if (!a.bias) {  // the two best logits' scores (softmax: up to the common denominator)
        g = a.sigmoid ? sigmoid_d(g) : exp(g - (double)m);
        if (g2 > -INFINITY) g2 = a.sigmoid ? sigmoid_d(g2) : exp(g2 - (double)m);
      }
      if (g2 > -INFINITY) g += g2;
    }
    int ahead = 0;  // groups ranked before this lane's
    for (int h = 0; h < a.n_group; ++h) {
      const double o = __shfl(g, h);
      ahead += (o > g || (o == g && h < lane)) ? 1 : 0;
    }
    const unsigned long long kept = __ballot(lane < a.n_group && ahead < a.topk_group);
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      const int e = lane + i * kWave;
      if (e < E && !((kept >> group_of(e, magic)) & 1)) key[i] = -INFINITY;
    }
  }

  int sel = -1;
  float sl = 0.f;
  for (int j = 0; j < a.k; ++j) {
    double bv = -INFINITY;
    int bi = 0x7fffffff;
#pragma unroll
    for (int i = 0; i < PL; ++i)
      if (key[i] > bv) {
        bv = key[i];
        bi = lane + i * kWave;
      }
    const double top = wave_max_d(bv);
    if (top == -INFINITY) break;  // wave-uniform: no expert is left
    bi = wave_min_i(bv == top ? bi : 0x7fffffff);
    float lw = 0.f;
#pragma unroll
    for (int i = 0; i < PL; ++i)
      if (lane + i * kWave == bi) {
        key[i] = -INFINITY;
        lw = l[i];
      }
    lw = __shfl(lw, bi & 63);
    if (lane == j) {
      sel = bi;
      sl = lw;
    }
  }
  const float w = gate_weight(lane, a.k, sel, sl, m, z, a.sigmoid, a.renormalize, a.scale);
  if (live && lane < a.k) {
    a.idx[t * a.k + lane] = sel;
    a.w[t * a.k + lane] = w;
  }
}

// ---------------------------------------------------------------------------
// Gradient of the gate weights
// ---------------------------------------------------------------------------
template <int PL>
__global__ __launch_bounds__(kTokens* kWave) void route_grouped_backward_kernel(RouteBwdArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * kTokens + (threadIdx.x >> 6);
  if (t >= a.T) return;  // whole wave exits together
  const int E = a.E, k = a.k;
  const float* row = a.logits + t * E;
  int id = -1;
  float g = 0.f, l = -INFINITY;
  if (lane < k) {
    id = a.idx[t * k + lane];
    if (id < 0 || id >= E) id = -1;
    if (id >= 0) {
      g = a.scale * a.d_w[t * k + lane];
      const float v = row[id];
      l = fminf(v, FLT_MAX);
      if (!(v > -INFINITY)) id = -1;  // an expert that is not available has score 0
    }
  }
  const bool has = id >= 0;
  const bool dense = !a.sigmoid && !a.renormalize;
  float d = 0.f, rest = 0.f, m = 0.f, z = 1.f;
  float x[PL];
  if (dense) {
    m = -FLT_MAX;
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      const int e = lane + i * kWave;
      const float v = e < E ? row[e] : -INFINITY;
      x[i] = v > -INFINITY ? fminf(v, FLT_MAX) : -INFINITY;
      m = fmaxf(m, x[i]);
    }
    m = wave_max_f(m);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      x[i] = expf(x[i] - m);
      s += x[i];
    }
    z = wave_sum_f(s);
    if (!(z > 0.f)) z = 1.f;  // no expert is available: every term is zero
    d = has ? g * (expf(l - m) / z) : 0.f;
    rest = wave_sum_f(d);
  } else if (a.renormalize) {
    float top = wave_max_f(has ? l : -FLT_MAX);
    if (a.sigmoid) top = fminf(top, 0.f);
    float s = 0.f;
    if (has) s = a.sigmoid ? expf(fminf(l, 0.f) - top) / (1.f + expf(-fabsf(l))) : expf(l - top);
    const float sum = wave_sum_f(s);
    const float q = has ? s / sum : 0.f;
    d = q * (g - wave_sum_f(has ? q * g : 0.f));
    if (a.sigmoid && has) d *= 1.f / (1.f + expf(l));  // 1 - s
  } else if (has) {
    const float s = 1.f / (1.f + expf(-l));
    d = g * s * (1.f / (1.f + expf(l)));
  }
  float o[PL];
#pragma unroll
  for (int i = 0; i < PL; ++i) o[i] = dense ? -(x[i] / z) * rest : 0.f;
  for (int j = 0; j < k; ++j) {
    const int e = __shfl(id, j);
    const float v = __shfl(d, j);
#pragma unroll
    for (int i = 0; i < PL; ++i)
      if (lane + i * kWave == e) o[i] += v;
  }
#pragma unroll
  for (int i = 0; i < PL; ++i)
    if (lane + i * kWave < E) a.d_logits[t * E + lane + i * kWave] = o[i];
}

}  // namespace

hipError_t launch_route_grouped(const RouteArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)((a.T + kTokens - 1) / kTokens)), block(kTokens * kWave);
  const int Eg = a.E / a.n_group;
  const uint32_t magic = ((1u << 22) + Eg - 1) / Eg;
  const size_t lds = a.n_group > 1 ? (size_t)kTokens * a.E * sizeof(double) : 0;
  const int pl = (a.E + kWave - 1) / kWave;
#define MOE_ROUTE(PL_) hipLaunchKernelGGL(route_grouped_kernel<PL_>, grid, block, lds, s, a, magic)
  if (pl <= 1) MOE_ROUTE(1);
  else if (pl <= 2) MOE_ROUTE(2);
  else if (pl <= 4) MOE_ROUTE(4);
  else if (pl <= 8) MOE_ROUTE(8);
  else MOE_ROUTE(16);
#undef MOE_ROUTE
  return hipGetLastError();
}

hipError_t launch_route_grouped_backward(const RouteBwdArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)((a.T + kTokens - 1) / kTokens)), block(kTokens * kWave);
  const int pl = (a.E + kWave - 1) / kWave;
#define MOE_ROUTE(PL_) hipLaunchKernelGGL(route_grouped_backward_kernel<PL_>, grid, block, 0, s, a)
  if (pl <= 1) MOE_ROUTE(1);
  else if (pl <= 2) MOE_ROUTE(2);
  else if (pl <= 4) MOE_ROUTE(4);
  else if (pl <= 8) MOE_ROUTE(8);
  else MOE_ROUTE(16);
#undef MOE_ROUTE
  return hipGetLastError();
}

}  // namespace moe
