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

constexpr int kTokens = 4;  // wavefronts per block

// Orders one wavefront's LDS accesses across its lanes (no instruction: they complete in issue order).
__device__ __forceinline__ void wave_lds_order() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// One token by one wavefront, with 64-bit keys throughout; lane l holds experts l, l + 64, ...  sk: E doubles of LDS
// of this wavefront's own (used when groups are dropped).
template <int PL>
__device__ void route_exact(const RouteArgs& a, int64_t t, int lane, uint32_t magic, double* sk) {
  const int E = a.E;
  float l[PL];
  double key[PL];
  bool ok[PL];
  float m = -FLT_MAX;
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    const int e = lane + i * kWave;
    const float v = (e < E) ? a.logits[t * E + e] : -INFINITY;
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
    const int Eg = E / a.n_group;
#pragma unroll
    for (int i = 0; i < PL; ++i)
      if (lane + i * kWave < E) sk[lane + i * kWave] = key[i];
    wave_lds_order();
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
  if (lane < a.k) {
    a.idx[t * a.k + lane] = sel;
    a.w[t * a.k + lane] = w;
  }
}

template <int PL>
__global__ __launch_bounds__(kTokens* kWave) void route_exact_kernel(RouteArgs a, uint32_t magic) {
  extern __shared__ double s_key[];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int64_t t = (int64_t)blockIdx.x * kTokens + wv;
  if (t < a.T) route_exact<PL>(a, t, lane, magic, s_key + wv * a.E);  // wave-uniform
}

// ---------------------------------------------------------------------------
// fp32 keys with a check: LT lanes per token, 64 / LT tokens per wavefront
// ---------------------------------------------------------------------------
// Reductions over the LT lanes of a token, result in every lane: the four steps inside a row of 16 lanes by DPP
// (quad swaps, half mirror, mirror), the rows of a 64-lane token by readlane.
template <int CTRL>
__device__ __forceinline__ float dppf(float v) {
  const int x = __builtin_bit_cast(int, v);
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(x, x, CTRL, 0xF, 0xF, false));
}
__device__ __forceinline__ float lanef(float v, int l) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), l));
}
template <int LT, typename F>
__device__ __forceinline__ float reduce(float v, F f) {
  v = f(v, dppf<0xB1>(v));
  v = f(v, dppf<0x4E>(v));
  v = f(v, dppf<0x141>(v));
  v = f(v, dppf<0x140>(v));
  if constexpr (LT == 64) v = f(f(lanef(v, 0), lanef(v, 16)), f(lanef(v, 32), lanef(v, 48)));
  return v;
}
template <int LT>
__device__ __forceinline__ float max_of(float v) {
  return reduce<LT>(v, [](float a, float b) { return fmaxf(a, b); });
}
template <int LT>
__device__ __forceinline__ float sum_of(float v) {
  return reduce<LT>(v, [](float a, float b) { return a + b; });
}

// 1 / (1 + e^-z) and e^z with the hardware exp2 and reciprocal (about 1 ulp each).
__device__ __forceinline__ float exp_fast(float z) { return __builtin_amdgcn_exp2f(z * 1.4426950408889634f); }
__device__ __forceinline__ float sigmoid_fast(float z) { return __builtin_amdgcn_rcpf(1.0f + exp_fast(-z)); }

// Compare-exchange network of a descending sort (Batcher's odd-even merge sort), N a power of two.
template <int N, typename F>
__device__ __forceinline__ void sort_network(F swap) {
#pragma unroll
  for (int p = 1; p < N; p *= 2)
#pragma unroll
    for (int q = p; q >= 1; q /= 2)
#pragma unroll
      for (int j = q % p; j + q < N; j += 2 * q)
#pragma unroll
        for (int i = 0; i < q; ++i)
          if (j + i + q < N && (j + i) / (2 * p) == (j + i + q) / (2 * p)) swap(j + i, j + i + q);
}

// Each group of E / n_group experts sits on LG = 2^lg_bits lanes, PL experts a lane, in order.  The best of a lane
// are sorted in registers, so a round of the selection is a maximum over the lanes' heads.
//
// Keys are fp32: logits without a bias (exact), else score + bias, off by at most delta = 1.25e-6 + 2.4e-7 max |key|
// (score: exp2 and reciprocal 1 ulp each, their argument's rounding passes on at most 0.23 of it, the softmax's
// common denominator moves all scores together; bias: one rounding).  Where the choice could come out differently
// within that -- two keys in a row within 2 delta (equal logits, whose order is by id, among them), or the last kept
// and the first dropped group within 5 delta -- the token goes to route_exact.  For scores spread over (0, 1) that
// is a few tokens in a thousand; 64-bit keys throughout cost 45 us at 16384 x 256 against REPLACE_US.
template <int LT, int PL, int PX>
__global__ __launch_bounds__(kTokens* kWave) void route_grouped_kernel(RouteArgs a, uint32_t magic, int n_group,
                                                                       int lg_bits, bool vec4) {
  extern __shared__ double s_key[];
  __shared__ int s_id[kTokens][64 / LT][32];
  constexpr int TPW = 64 / LT;
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, l = lane & (LT - 1), sub = lane / LT;
  const int64_t t0 = ((int64_t)blockIdx.x * kTokens + wv) * TPW, t = t0 + sub;
  const bool live = t < a.T;
  const int E = a.E, Eg = E / n_group, k = a.k;
  const int g = l >> lg_bits, s0 = (l & ((1 << lg_bits) - 1)) * PL;  // this lane's group, first expert in it
  const int e0 = g * Eg + s0, ne = (live && g < n_group) ? min(PL, Eg - s0) : 0;  // (negative: none)
  const float* row = a.logits + t * E;
  float x[PL], key[PL];
  int id[PL];
  if (vec4 && ne == PL && PL % 4 == 0) {
#pragma unroll
    for (int i = 0; i < PL; i += 4) {
      const floatx4 v = *reinterpret_cast<const floatx4*>(row + e0 + i);
#pragma unroll
      for (int q = 0; q < 4 && i + q < PL; ++q) x[i + q] = v[q];
    }
  } else {
#pragma unroll
    for (int i = 0; i < PL; ++i) x[i] = i < ne ? row[e0 + i] : -INFINITY;
  }
  float m = -FLT_MAX;
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    id[i] = e0 + i;
    x[i] = x[i] > -INFINITY ? fminf(x[i], FLT_MAX) : -INFINITY;  // NaN: not available
  }
  float b[PL];
  if (a.bias) {
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      b[i] = i < ne ? a.bias[e0 + i] : 0.f;
      if (!(b[i] > -INFINITY)) x[i] = -INFINITY;
      b[i] = fminf(b[i], FLT_MAX);
    }
  }
  float z = 1.f;
  if (!a.sigmoid) {
#pragma unroll
    for (int i = 0; i < PL; ++i) m = fmaxf(m, x[i]);
    m = max_of<LT>(m);
    if (a.bias || !a.renormalize) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < PL; ++i) s += exp_fast(x[i] - m);
      z = sum_of<LT>(s);
    }
  }
  auto score = [&](float v) { return a.sigmoid ? sigmoid_fast(v) : exp_fast(v - m) / z; };
  float delta = 0.f;
  if (a.bias) {
    float big = 0.f;
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      const bool ok = x[i] > -INFINITY;
      key[i] = ok ? score(x[i]) + b[i] : -INFINITY;
      big = fmaxf(big, ok ? fabsf(key[i]) : 0.f);
    }
    delta = 1.25e-6f + 2.4e-7f * max_of<LT>(big);
  } else {
#pragma unroll
    for (int i = 0; i < PL; ++i) key[i] = x[i];
  }
  sort_network<PL>([&](int i, int j) {
    const bool swap = key[j] > key[i];
    const float ki = key[i];
    const int ii = id[i];
    key[i] = swap ? key[j] : ki;
    key[j] = swap ? ki : key[j];
    id[i] = swap ? id[j] : ii;
    id[j] = swap ? ii : id[j];
  });

  bool unsure = false;
  if (n_group > 1) {  // the launcher passes one group where all are kept
    float g1 = key[0], g2 = PL > 1 ? key[PL > 1 ? 1 : 0] : -INFINITY;
    auto merge = [&](float o1, float o2) {
      g2 = fmaxf(fminf(g1, o1), fmaxf(g2, o2));
      g1 = fmaxf(g1, o1);
    };
    if (lg_bits >= 1) merge(dppf<0xB1>(g1), dppf<0xB1>(g2));
    if (lg_bits >= 2) merge(dppf<0x4E>(g1), dppf<0x4E>(g2));
    if (lg_bits >= 3) merge(dppf<0x141>(g1), dppf<0x141>(g2));
    if (lg_bits >= 4) merge(dppf<0x140>(g1), dppf<0x140>(g2));
    if (LT == 64 && lg_bits >= 5) merge(__shfl_xor(g1, 16), __shfl_xor(g2, 16));
    float gd = delta;
    if (a.group_top == 2) {
      if (!a.bias) {
        gd = 1.5e-6f;
        g1 = g1 > -INFINITY ? score(g1) : g1;
        g2 = g2 > -INFINITY ? score(g2) : g2;
      }
      if (g2 > -INFINITY) g1 += g2;
    }
    int ahead = 0;  // lanes of better groups
    if constexpr (LT == 16) {
#define MOE_ROR(N) ahead += dppf<0x120 + N>(g1) > g1 ? 1 : 0;
      MOE_ROR(1) MOE_ROR(2) MOE_ROR(3) MOE_ROR(4) MOE_ROR(5) MOE_ROR(6) MOE_ROR(7) MOE_ROR(8)
      MOE_ROR(9) MOE_ROR(10) MOE_ROR(11) MOE_ROR(12) MOE_ROR(13) MOE_ROR(14) MOE_ROR(15)
#undef MOE_ROR
    } else {
      for (int h = 0; h < n_group; ++h) ahead += (lanef(g1, h << lg_bits) > g1 ? 1 : 0) << lg_bits;
    }
    const bool keep = ahead < (a.topk_group << lg_bits);
    // Lanes of no group hold -inf and are ahead of nothing.
    const float low = -max_of<LT>(keep && g1 > -INFINITY ? -g1 : -INFINITY), high = max_of<LT>(keep ? -INFINITY : g1);
    unsure = low - high <= 5.f * gd;
    // Equal groups can leave more than topk_group kept (none is ahead of the other).
    const float kept = sum_of<LT>(keep && g1 > -INFINITY ? 1.f : 0.f);
    unsure = unsure || kept > (float)(a.topk_group << lg_bits);
    if (!keep)
#pragma unroll
      for (int i = 0; i < PL; ++i) key[i] = -INFINITY;
  }

  int* ids = s_id[wv][sub];
  if (l < k) ids[l] = -1;
  wave_lds_order();
  float prev = INFINITY;
  const float tol = 2.f * delta;
  for (int j = 0; j <= k; ++j) {  // one round more than slots: the first that misses has to miss clearly
    const float top = max_of<LT>(key[0]);
    unsure = unsure || (top > -INFINITY && prev - top <= tol);
    prev = top;
    if (j == k) break;
    const unsigned long long at = __ballot(key[0] == top && top > -INFINITY);
    const uint32_t mine = LT == 64 ? 0 : (uint32_t)(at >> (lane & 48)) & 0xffffu;
    const bool win = LT == 64 ? at != 0 && lane == __builtin_ctzll(at) : mine != 0 && l == __builtin_ctz(mine);
    if (win) {
      ids[j] = id[0];
#pragma unroll
      for (int i = 0; i + 1 < PL; ++i) {
        key[i] = key[i + 1];
        id[i] = id[i + 1];
      }
      key[PL - 1] = -INFINITY;
    }
  }
  wave_lds_order();
  // Slot j's id on lane j (k <= LT).
  const int sel = l < k ? ids[l] : -1;
  const bool has = live && sel >= 0;
  const float sl = has ? fminf(row[sel], FLT_MAX) : 0.f;
  float s = 0.f, w = 0.f;
  if (a.renormalize) {
    float top = max_of<LT>(has ? sl : -FLT_MAX);
    if (a.sigmoid) top = fminf(top, 0.f);
    if (has) s = a.sigmoid ? expf(fminf(sl, 0.f) - top) / (1.f + expf(-fabsf(sl))) : expf(sl - top);
    const float sum = sum_of<LT>(s);
    w = has ? a.scale * (s / sum) : 0.f;
  } else if (has) {
    w = a.scale * (a.sigmoid ? 1.f / (1.f + expf(-sl)) : expf(sl - m) / z);
  }
  const unsigned long long doubt = __ballot(unsure && live);
  const bool mine_sure = LT == 64 ? doubt == 0 : ((doubt >> (lane & 48)) & 0xffffu) == 0;
  if (live && l < k && mine_sure) {
    a.idx[t * k + l] = sel;
    a.w[t * k + l] = w;
  }
  if (doubt != 0)
    for (int q = 0; q < TPW; ++q)
      if (LT == 64 || ((doubt >> (16 * q)) & 0xffffu) != 0)
        route_exact<PX>(a, t0 + q, lane, magic, s_key + wv * E);
}

// ---------------------------------------------------------------------------
// Gradient of the gate weights
// ---------------------------------------------------------------------------
// HBM-bound: reads the chosen logits (the plain softmax's gradient: all of them), writes every gradient once.  LT
// lanes per token; lane l holds V consecutive experts (4: 16-byte accesses, E % 4 == 0) from V (l + LT i), i < PL.
// The chosen experts' terms are handed to the lanes that hold them one by one, so that repeated ids add up in order.
template <int LT, int V, int PL>
__global__ __launch_bounds__(kTokens* kWave) void route_grouped_backward_kernel(RouteBwdArgs a) {
  const int lane = threadIdx.x & 63, l = lane & (LT - 1);
  const int64_t t = ((int64_t)blockIdx.x * kTokens + (threadIdx.x >> 6)) * (64 / LT) + lane / LT;
  const bool live = t < a.T;
  const int E = a.E, k = a.k;
  const float* row = a.logits + t * E;
  int id = -1;
  float g = 0.f, lg = -INFINITY;
  if (live && l < k) {
    id = a.idx[t * k + l];
    g = a.scale * a.d_w[t * k + l];
    if (id < 0 || id >= E) id = -1;
    if (id >= 0) {
      const float v = row[id];
      lg = fminf(v, FLT_MAX);
      if (!(v > -INFINITY)) id = -1;  // an expert that is not available has score 0
    }
  }
  const bool has = id >= 0;
  const bool dense = !a.sigmoid && !a.renormalize;
  float o[PL][V];
  float d = 0.f;
  if (dense) {
    float m = -FLT_MAX;
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      const int e = V * (l + LT * i);
#pragma unroll
      for (int q = 0; q < V; ++q) o[i][q] = -INFINITY;
      if (live && e < E) {
        if constexpr (V == 4) {
          const floatx4 v = *reinterpret_cast<const floatx4*>(row + e);
#pragma unroll
          for (int q = 0; q < 4; ++q) o[i][q] = v[q];
        } else {
          o[i][0] = row[e];
        }
      }
#pragma unroll
      for (int q = 0; q < V; ++q) {
        o[i][q] = o[i][q] > -INFINITY ? fminf(o[i][q], FLT_MAX) : -INFINITY;
        m = fmaxf(m, o[i][q]);
      }
    }
    m = max_of<LT>(m);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < PL; ++i)
#pragma unroll
      for (int q = 0; q < V; ++q) {
        o[i][q] = exp_fast(o[i][q] - m);
        s += o[i][q];
      }
    float z = sum_of<LT>(s);
    z = z > 0.f ? 1.f / z : 0.f;  // no expert is available: every term is zero
    d = has ? g * (exp_fast(lg - m) * z) : 0.f;
    const float rest = sum_of<LT>(d) * z;
#pragma unroll
    for (int i = 0; i < PL; ++i)
#pragma unroll
      for (int q = 0; q < V; ++q) o[i][q] *= -rest;
  } else {
    if (a.renormalize) {
      float top = max_of<LT>(has ? lg : -FLT_MAX);
      if (a.sigmoid) top = fminf(top, 0.f);
      float s = 0.f;
      if (has) s = a.sigmoid ? expf(fminf(lg, 0.f) - top) / (1.f + expf(-fabsf(lg))) : expf(lg - top);
      const float sum = sum_of<LT>(s);
      const float q = has ? s / sum : 0.f;
      d = q * (g - sum_of<LT>(has ? q * g : 0.f));
      if (a.sigmoid && has) d *= 1.f / (1.f + expf(lg));  // 1 - s
    } else if (has) {
      d = g * (1.f / (1.f + expf(-lg))) * (1.f / (1.f + expf(lg)));
    }
#pragma unroll
    for (int i = 0; i < PL; ++i)
#pragma unroll
      for (int q = 0; q < V; ++q) o[i][q] = 0.f;
  }
  if (!has) d = 0.f;
  for (int j = 0; j < k; ++j) {
    const int e = LT == 64 ? __builtin_amdgcn_readlane(id, j) : __shfl(id, (lane & 48) + j);
    const float v = LT == 64 ? lanef(d, j) : __shfl(d, (lane & 48) + j);
#pragma unroll
    for (int i = 0; i < PL; ++i)
#pragma unroll
      for (int q = 0; q < V; ++q) o[i][q] += V * (l + LT * i) + q == e ? v : 0.f;
  }
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    const int e = V * (l + LT * i);
    if (live && e < E) {
      if constexpr (V == 4)
        __builtin_nontemporal_store(floatx4{o[i][0], o[i][1], o[i][2], o[i][3]}, reinterpret_cast<floatx4*>(a.d_logits + t * E + e));
      else
        a.d_logits[t * E + e] = o[i][0];
    }
  }
}

}  // namespace

hipError_t launch_route_grouped(const RouteArgs& a, hipStream_t s) {
  const int n_group = a.topk_group < a.n_group ? a.n_group : 1;  // groups restrict the choice only if some are dropped
  const int Eg = a.E / n_group;
  const uint32_t magic = ((1u << 22) + a.E / a.n_group - 1) / (a.E / a.n_group);
  const size_t lds = n_group > 1 ? (size_t)kTokens * a.E * sizeof(double) : 0;
  auto lanes_per_group = [&](int lt) {  // log2, or -1
    if (n_group > lt) return -1;
    int bits = 0;
    while (n_group << (bits + 1) <= lt) ++bits;
    return bits;
  };
  auto per_lane = [&](int bits) { return bits < 0 ? 1 << 20 : (Eg + (1 << bits) - 1) >> bits; };
  const int b16 = lanes_per_group(16), b64 = lanes_per_group(64), p16 = per_lane(b16), p64 = per_lane(b64);
  const int px = (a.E + kWave - 1) / kWave;
  const bool aligned = a.E % 4 == 0 && Eg % 4 == 0;
  // 16 lanes a token share the rounds of the selection between four tokens; 64 have fewer experts a lane to sort,
  // which is quicker until the tokens fill the chip.
  if (p16 <= 16 && a.k <= 16 && (p16 <= 4 || a.T > 2048)) {
    const dim3 grid((unsigned)((a.T + 4 * kTokens - 1) / (4 * kTokens))), block(kTokens * kWave);
#define MOE_ROUTE(PL_, PX_) \
  hipLaunchKernelGGL((route_grouped_kernel<16, PL_, PX_>), grid, block, lds, s, a, magic, n_group, b16, aligned)
    if (p16 <= 1) MOE_ROUTE(1, 1);
    else if (p16 <= 2) MOE_ROUTE(2, 1);
    else if (p16 <= 4) MOE_ROUTE(4, 1);
    else if (p16 <= 8) MOE_ROUTE(8, 2);
    else MOE_ROUTE(16, 4);
#undef MOE_ROUTE
    return hipGetLastError();
  }
  const dim3 grid((unsigned)((a.T + kTokens - 1) / kTokens)), block(kTokens * kWave);
  if (p64 <= 8) {
#define MOE_ROUTE(PL_, PX_) \
  hipLaunchKernelGGL((route_grouped_kernel<64, PL_, PX_>), grid, block, lds, s, a, magic, n_group, b64, aligned)
    if (p64 <= 1) MOE_ROUTE(1, 1);
    else if (p64 <= 2) MOE_ROUTE(2, 2);
    else if (p64 <= 4) MOE_ROUTE(4, 4);
    else MOE_ROUTE(8, 8);
#undef MOE_ROUTE
    return hipGetLastError();
  }
#define MOE_ROUTE(PL_) hipLaunchKernelGGL(route_exact_kernel<PL_>, grid, block, lds, s, a, magic)
  if (px <= 4) MOE_ROUTE(4);
  else MOE_ROUTE(16);
#undef MOE_ROUTE
  return hipGetLastError();
}

hipError_t launch_route_grouped_backward(const RouteBwdArgs& a, hipStream_t s) {
  const dim3 block(kTokens * kWave);
  const auto grid = [&](int per_wave) { return dim3((unsigned)((a.T + per_wave * kTokens - 1) / (per_wave * kTokens))); };
#define MOE_ROUTE(LT_, V_, PL_) \
  hipLaunchKernelGGL((route_grouped_backward_kernel<LT_, V_, PL_>), grid(64 / LT_), block, 0, s, a)
  if (a.E % 4 == 0) {
    if (a.E <= 64 && a.k <= 16) MOE_ROUTE(16, 4, 1);
    else if (a.E <= 256) MOE_ROUTE(64, 4, 1);
    else if (a.E <= 512) MOE_ROUTE(64, 4, 2);
    else MOE_ROUTE(64, 4, 4);
  } else {
    if (a.E <= 64) MOE_ROUTE(64, 1, 1);
    else if (a.E <= 256) MOE_ROUTE(64, 1, 4);
    else MOE_ROUTE(64, 1, 16);
  }
#undef MOE_ROUTE
  return hipGetLastError();
}

}  // namespace moe
