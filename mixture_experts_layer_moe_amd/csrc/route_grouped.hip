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
// and sums of two scores are 64-bit: with logits of full fp32 precision two of
// them that differ by less than an fp32 rounding are met every few thousand
// tokens.
//
// Bound by instruction issue once the tokens fill the chip: 16384 x 256, 8 of 4
// of 8 groups, takes 16-17 us (the logits alone would take 3.5).  1300 VALU
// instructions a wavefront, four wavefronts a SIMD: its VALU is busy for 97 % of
// an average wavefront's life and 68 % of the launch, whose last 3-4 us are the
// few tokens that are chosen again in 64 bits.  With a wavefront a SIMD or less
// bound by the chain of dependent steps (sort, groups, k rounds): 4099 x 160 6-8
// us (VALU 34 %), one token 4.7-5.5 (25 %), of which a launch is 2.3.
// Where ties are common most tokens are chosen again: 16384 x 256 with bf16
// logits 26 us without a bias and 34 with one of zeros, with two experts pushed
// out by a bias of -1e9 37 (the doubt test's tolerance goes by the row's largest
// key); 4099 x 160 with bf16 logits or masks of -1e4 and below 15-16.
#include "operators.h"

#include <float.h>

namespace moe {
namespace {

constexpr int kTokens = 4;  // wavefronts per block

// Orders one wavefront's LDS accesses across its lanes (no instruction: they complete in issue order).
__device__ __forceinline__ void wave_lds_order() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Values of another lane: by DPP inside a row of 16 lanes, or of a given lane.
template <int CTRL>
__device__ __forceinline__ int dpp(int x) {
  return __builtin_amdgcn_update_dpp(x, x, CTRL, 0xF, 0xF, false);
}
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __builtin_bit_cast(float, dpp<CTRL>(__builtin_bit_cast(int, v)));
}
template <int CTRL>
__device__ __forceinline__ double dpp(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)dpp<CTRL>((int)(uint32_t)u), hi = (uint32_t)dpp<CTRL>((int)(u >> 32));
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ float of_lane(float v, int l) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), l));
}
__device__ __forceinline__ double of_lane(double v, int l) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, l);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(u >> 32), l);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// Reductions over the LT lanes of a token, result in every lane: four steps inside a row of 16 lanes (quad swaps,
// half mirror, mirror), then the four rows of a 64-lane token.
template <int LT, typename K, typename F>
__device__ __forceinline__ K reduce(K v, F f) {
  v = f(v, dpp<0xB1>(v));
  v = f(v, dpp<0x4E>(v));
  v = f(v, dpp<0x141>(v));
  v = f(v, dpp<0x140>(v));
  if constexpr (LT == 64) v = f(f(of_lane(v, 0), of_lane(v, 16)), f(of_lane(v, 32), of_lane(v, 48)));
  return v;
}
__device__ __forceinline__ float max2(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ double max2(double a, double b) { return fmax(a, b); }
__device__ __forceinline__ float min2(float a, float b) { return fminf(a, b); }
__device__ __forceinline__ double min2(double a, double b) { return fmin(a, b); }
template <int LT, typename K>
__device__ __forceinline__ K max_of(K v) {
  return reduce<LT>(v, [](K a, K b) { return max2(a, b); });
}
template <int LT, typename K>
__device__ __forceinline__ K sum_of(K v) {
  return reduce<LT>(v, [](K a, K b) { return a + b; });
}

// e^z from the hardware exp2, with the rounding of z / ln 2 carried along: about 2 ulp whatever z.
__device__ __forceinline__ float exp_of(float z) {
  z = __builtin_amdgcn_fmed3f(z, -200.f, 100.f);  // (0 and infinity already)
  const float t = z * 1.4426950408889634f;
  return __builtin_amdgcn_exp2f(t) * fmaf(fmaf(z, 1.4426950408889634f, -t), 0.69314718055994531f, 1.f);
}
__device__ __forceinline__ float inverse(float v) { return __builtin_amdgcn_rcpf(v); }
// 1 / (1 + e^-z)
__device__ __forceinline__ float sigmoid_of(float z) { return inverse(1.f + exp_of(-z)); }

// Scaled score of a chosen logit for renormalised weights: both scores times a common factor that keeps the largest
// of the row at least 1/2: softmax e^(l - top), sigmoid(l) = e^min(l, 0) / (1 + e^-|l|) with e^min(l, 0) scaled by
// e^-top, top = min(largest chosen logit, 0).
__device__ __forceinline__ float scaled_score(bool sigmoid, float l, float top) {
  return sigmoid ? exp_of(fminf(l, 0.f) - top) * inverse(1.f + exp_of(-fabsf(l))) : exp_of(l - top);
}

// Compare-exchange network of a sort (Batcher's odd-even merge sort), N a power of two.
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

// Where a lane's experts lie: each group of Eg = E / n_group experts sits on 2^lg_bits lanes, PL experts a lane, in
// order (n_group is 1 where no group is dropped).
struct Place {
  int n_group, lg_bits;
  bool vec4;  // rows and groups are whole 16-byte pieces
};

// Ranks a lane's group among the others: the number of lanes of better groups, `better(o, mine, h)` saying whether
// group h of sum o comes ahead.
template <int LT, typename K, typename F>
__device__ __forceinline__ int lanes_ahead(const Place& pl, K sum, F better) {
  int ahead = 0;
  if constexpr (LT == 16) {
#define MOE_ROR(N) ahead += better(dpp<0x120 + N>(sum), sum, -1) ? 1 : 0;
    MOE_ROR(1) MOE_ROR(2) MOE_ROR(3) MOE_ROR(4) MOE_ROR(5) MOE_ROR(6) MOE_ROR(7) MOE_ROR(8)
    MOE_ROR(9) MOE_ROR(10) MOE_ROR(11) MOE_ROR(12) MOE_ROR(13) MOE_ROR(14) MOE_ROR(15)
#undef MOE_ROR
  } else {
    for (int h = 0; h < pl.n_group; ++h)
      ahead += (better(of_lane(sum, h << pl.lg_bits), sum, h) ? 1 : 0) << pl.lg_bits;
  }
  return ahead;
}

// The two largest keys of a group, from each lane's two largest.
template <int LT, typename K>
__device__ __forceinline__ void group_best(const Place& pl, K& g1, K& g2) {
  auto merge = [&](K o1, K o2) {
    g2 = max2(min2(g1, o1), max2(g2, o2));
    g1 = max2(g1, o1);
  };
  if (pl.lg_bits >= 1) merge(dpp<0xB1>(g1), dpp<0xB1>(g2));
  if (pl.lg_bits >= 2) merge(dpp<0x4E>(g1), dpp<0x4E>(g2));
  if (pl.lg_bits >= 3) merge(dpp<0x141>(g1), dpp<0x141>(g2));
  if (pl.lg_bits >= 4) merge(dpp<0x140>(g1), dpp<0x140>(g2));
  if (LT == 64 && pl.lg_bits >= 5) merge(__shfl_xor(g1, 16), __shfl_xor(g2, 16));
}

// The lane of the token's LT lanes that takes a round: the first whose head is the largest key; false if none is left.
template <int LT>
__device__ __forceinline__ bool wins(bool head, int l, int lane) {
  const unsigned long long at = __ballot(head);
  if constexpr (LT == 64) return at != 0 && lane == __builtin_ctzll(at);
  const uint32_t mine = (uint32_t)(at >> (lane & 48)) & 0xffffu;
  return mine != 0 && l == __builtin_ctz(mine);
}

// Chooses the k experts of a token held by a wavefront into ids[0, k) (-1: none) by 64-bit keys, equal ones lowest id
// first.  x: this lane's logits (-inf: not available), m: the row's largest (softmax).
template <int PL>
__device__ void choose_exact(const RouteArgs& a, const Place& pl, int lane, int e0, const float (&x)[PL],
                             const float (&b)[PL], float m, int* ids) {
  const double none = -INFINITY;
  double key[PL];
  int id[PL];
  double iz = 1.0;
  if (!a.sigmoid && a.bias) {
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < PL; ++i) s += x[i] > -INFINITY ? exp((double)x[i] - (double)m) : 0.0;
    iz = 1.0 / sum_of<64>(s);
  }
  auto score = [&](double v) { return a.sigmoid ? 1.0 / (1.0 + exp(-v)) : exp(v - (double)m) * iz; };
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    id[i] = e0 + i;
    key[i] = !a.bias ? (double)x[i] : x[i] > -INFINITY ? score(x[i]) + (double)b[i] : none;
  }
  sort_network<PL>([&](int i, int j) {
    const bool swap = key[j] > key[i] || (key[j] == key[i] && id[j] < id[i]);
    const double ki = key[i];
    const int ii = id[i];
    key[i] = swap ? key[j] : ki;
    key[j] = swap ? ki : key[j];
    id[i] = swap ? id[j] : ii;
    id[j] = swap ? ii : id[j];
  });
  if (pl.n_group > 1) {
    double g1 = key[0], g2 = PL > 1 ? key[PL > 1 ? 1 : 0] : none;
    group_best<64>(pl, g1, g2);
    if (a.group_top == 2) {
      if (!a.bias) {
        g1 = g1 > none ? score(g1) : g1;
        g2 = g2 > none ? score(g2) : g2;
      }
      if (g2 > none) g1 += g2;
    }
    const int mine = lane >> pl.lg_bits;
    const int ahead = lanes_ahead<64>(pl, g1, [&](double o, double g, int h) { return o > g || (o == g && h < mine); });
    if (ahead >= (a.topk_group << pl.lg_bits))
#pragma unroll
      for (int i = 0; i < PL; ++i) key[i] = none;
  }
  if (lane < a.k) ids[lane] = -1;
  wave_lds_order();
  for (int j = 0; j < a.k; ++j) {
    const double top = max_of<64>(key[0]);
    if (wins<64>(key[0] == top && top > none, lane, lane)) {
      ids[j] = id[0];
#pragma unroll
      for (int i = 0; i + 1 < PL; ++i) {
        key[i] = key[i + 1];
        id[i] = id[i + 1];
      }
      key[PL - 1] = none;
    }
  }
  wave_lds_order();
}

// e^z and 1 / (1 + e^-z) by the hardware exp2 and reciprocal alone; z's rounding passes on at most 1.5e-8 of either
// score, so both are within 5e-7.
__device__ __forceinline__ float exp_fast(float z) { return __builtin_amdgcn_exp2f(z * 1.4426950408889634f); }
__device__ __forceinline__ float sigmoid_fast(float z) { return __builtin_amdgcn_rcpf(1.f + exp_fast(-z)); }

// The same for a token held by LT lanes, by fp32 keys; returns whether they leave the choice in doubt (then ids mean
// nothing).  z: sum of e^(l - m), for the plain softmax's weights.
//
// A key's last log2(PL) bits hold its place on the lane, so the lane's keys are sorted by maxima and minima alone
// (2 instructions an exchange; with the place beside it 5).  Keys (logits, or score + bias) are then off by at most
// delta = PL 2^-23 max |key|, with a bias 1.25e-6 + 2.4e-7 max |key| more: scores within 5e-7, the softmax's
// denominator 5e-7 of them, the sum's rounding.  Two keys in a row within 2 delta (equal ones, whose order is by id,
// among them), or the last kept and the first dropped group within 5 delta, leave the choice in doubt, and so does an
// available key next to the value that stands for none, or whose sum with another could be.
template <int LT, int PL>
__device__ __forceinline__ bool choose_fast(const RouteArgs& a, const Place& pl, int l, int lane, int e0, const float (&x)[PL],
                                            const float (&b)[PL], float m, int* ids, float& z) {
  constexpr uint32_t kPlace = PL - 1;
  constexpr float kNone = -3.402e38f, kLeast = -3.3e38f;  // no key; the least that is taken for one, or for a sum
  const int k = a.k;
  float key[PL];
  bool doubt = false;
  if (!a.sigmoid && (a.bias || !a.renormalize)) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < PL; ++i) s += exp_fast(x[i] - m);
    z = sum_of<LT>(s);
  }
  const float iz = a.sigmoid ? 1.f : inverse(z);
  auto score = [&](float v) { return a.sigmoid ? sigmoid_fast(v) : exp_fast(v - m) * iz; };
  float big = 0.f, least = INFINITY;
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    const bool ok = x[i] > -INFINITY;
    const float v = !a.bias ? x[i] : score(x[i]) + b[i];
    big = fmaxf(big, ok ? fabsf(v) : 0.f);
    least = ok ? fminf(least, v) : least;
    key[i] = __builtin_bit_cast(float, (__builtin_bit_cast(uint32_t, ok ? v : kNone) & ~kPlace) | (uint32_t)i);
  }
  doubt = least < (a.bias && a.group_top == 2 ? -1.6e38f : kLeast);  // (sums of two from -1.6e38 stay above kLeast)
  const float delta = max_of<LT>(big) * (PL * 1.1920929e-7f + (a.bias ? 2.4e-7f : 0.f)) + (a.bias ? 1.25e-6f : 0.f);
  sort_network<PL>([&](int i, int j) {
    const float hi = fmaxf(key[i], key[j]), lo = fminf(key[i], key[j]);
    key[i] = hi;
    key[j] = lo;
  });

  if (pl.n_group > 1) {
    float g1 = key[0], g2 = PL > 1 ? key[PL > 1 ? 1 : 0] : kNone;
    group_best<LT>(pl, g1, g2);
    float gd = delta;
    if (a.group_top == 2) {
      if (!a.bias) {
        // A score changes by no more than its logit does (softmax: below the row's largest; a place in a key's last
        // bits can lift it above, by whole units where logits are in the millions).
        gd += 1.5e-6f;
        auto group_score = [&](float v) { return score(a.sigmoid ? v : fminf(v, m)); };
        g1 = g1 > kLeast ? group_score(g1) : g1;
        g2 = g2 > kLeast ? group_score(g2) : g2;
      }
      g1 = g2 > kLeast ? g1 + g2 : g1;
    }
    g1 = g1 > kLeast ? g1 : -INFINITY;
    const int most = a.topk_group << pl.lg_bits;
    const bool keep = lanes_ahead<LT>(pl, g1, [](float o, float g, int) { return o > g; }) < most;
    // Lanes of no group are ahead of nothing.  Equal groups can leave more than topk_group kept.
    const bool in = keep && g1 > -INFINITY;
    const float low = -max_of<LT>(in ? -g1 : -INFINITY), high = max_of<LT>(keep ? -INFINITY : g1);
    const float kept = sum_of<LT>(in ? 1.f : 0.f);
    // (the last term: places alone, where keys are zeros or below the normal range)
    doubt = doubt || low - high <= 5.f * gd + 1e-37f || kept > (float)most;
    if (!keep)
#pragma unroll
      for (int i = 0; i < PL; ++i) key[i] = kNone;
  }

  if (l < k) ids[l] = -1;
  wave_lds_order();
  float prev = INFINITY;
  const float tol = 2.f * delta + 1e-37f;
  for (int j = 0; j <= k; ++j) {  // a round more than slots: the first that misses has to miss clearly
    const float top = max_of<LT>(key[0]);
    doubt = doubt || (top > kLeast && prev - top <= tol);
    prev = top;
    if (j == k) break;
    if (wins<LT>(key[0] == top && top > kLeast, l, lane)) {
      ids[j] = e0 + (int)(__builtin_bit_cast(uint32_t, top) & kPlace);
      constexpr int D = PL < 9 ? PL : 9;  // what lies deeper than k + 1 in a lane's list is not looked at
#pragma unroll
      for (int i = 0; i + 1 < D; ++i) key[i] = key[i + 1];
      if (PL > D && k > 8) {
#pragma unroll
        for (int i = D - 1; i + 1 < PL; ++i) key[i] = key[i + 1];
        key[PL - 1] = kNone;
      } else {
        key[D - 1] = kNone;
      }
    }
  }
  wave_lds_order();
  return doubt;
}

// This lane's logits and biases of token t: experts e0 .. of group l >> lg_bits.
template <int PL>
__device__ __forceinline__ int load_experts(const RouteArgs& a, const Place& pl, int64_t t, bool live, int l, float (&x)[PL],
                                            float (&b)[PL]) {
  const int Eg = a.E / pl.n_group, g = l >> pl.lg_bits, s0 = (l & ((1 << pl.lg_bits) - 1)) * PL;
  const int e0 = g * Eg + s0, ne = (live && g < pl.n_group) ? min(PL, Eg - s0) : 0;  // (negative: none)
  const float* row = a.logits + t * a.E;
  if (PL % 4 == 0 && pl.vec4 && ne == PL) {
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
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    x[i] = x[i] > -INFINITY ? fminf(x[i], FLT_MAX) : -INFINITY;  // NaN: not available
    b[i] = 0.f;
  }
  if (a.bias) {
    if (PL % 4 == 0 && pl.vec4 && ne == PL) {
#pragma unroll
      for (int i = 0; i < PL; i += 4) {
        const floatx4 v = *reinterpret_cast<const floatx4*>(a.bias + e0 + i);
#pragma unroll
        for (int q = 0; q < 4 && i + q < PL; ++q) b[i + q] = v[q];
      }
    } else {
#pragma unroll
      for (int i = 0; i < PL; ++i) b[i] = i < ne ? a.bias[e0 + i] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      if (!(b[i] > -INFINITY)) x[i] = -INFINITY;
      b[i] = fminf(b[i], FLT_MAX);
    }
  }
  return e0;
}

// This lane's share of the row's largest logit.
template <int LT, int PL>
__device__ __forceinline__ float row_max(const float (&x)[PL]) {
  float m = -FLT_MAX;
#pragma unroll
  for (int i = 0; i < PL; ++i) m = fmaxf(m, x[i]);
  return max_of<LT>(m);
}

// One token by a whole wavefront, in 64 bits.
template <int PL>
__device__ void choose_token(const RouteArgs& a, const Place& pl, int64_t t, int lane, int* ids) {
  float x[PL], b[PL];
  const int e0 = load_experts<PL>(a, pl, t, true, lane, x, b);
  choose_exact<PL>(a, pl, lane, e0, x, b, a.sigmoid ? 0.f : row_max<64>(x), ids);
}

// LT lanes per token, 64 / LT tokens per wavefront.  Tokens that fp32 keys leave in doubt are chosen again in 64 bits
// (PX experts a lane): at 16384 x 256 with normal fp32 logits a few in a thousand; 64-bit keys for all took 45 us there.
template <int LT, int PL, int PX>
__global__ __launch_bounds__(kTokens* kWave) void route_grouped_kernel(RouteArgs a, Place pl, int exact_bits) {
  __shared__ int s_id[kTokens][64 / LT][32];
  constexpr int TPW = 64 / LT;
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, l = lane & (LT - 1), sub = lane / LT;
  const int64_t t0 = ((int64_t)blockIdx.x * kTokens + wv) * TPW, t = t0 + sub;
  const bool live = t < a.T;
  float x[PL], b[PL], m = 0.f, z = 1.f;
  const int e0 = load_experts<PL>(a, pl, t, live, l, x, b);
  if (!a.sigmoid) m = row_max<LT>(x);
  int* ids = s_id[wv][sub];
  const bool doubt = choose_fast<LT, PL>(a, pl, l, lane, e0, x, b, m, ids, z);
  const unsigned long long again = __ballot(doubt && live);
  if (again != 0) {
    const Place px{pl.n_group, exact_bits, pl.vec4};
    for (int q = 0; q < TPW; ++q)
      if (LT == 64 || ((again >> (16 * q)) & 0xffffu) != 0) choose_token<PX>(a, px, t0 + q, lane, s_id[wv][q]);
  }
  // Slot j's id on lane j (k <= LT).
  const int sel = l < a.k ? ids[l] : -1;
  const bool has = live && sel >= 0;
  const float lg = has ? fminf(a.logits[t * a.E + sel], FLT_MAX) : 0.f;
  float w = 0.f;
  if (a.renormalize) {
    float top = max_of<LT>(has ? lg : -FLT_MAX);
    if (a.sigmoid) top = fminf(top, 0.f);
    const float s = has ? scaled_score(a.sigmoid, lg, top) : 0.f, sum = sum_of<LT>(s);
    w = has ? a.scale * (s * inverse(sum)) : 0.f;
  } else if (has) {
    w = a.scale * (a.sigmoid ? sigmoid_of(lg) : exp_of(lg - m) * inverse(z));
  }
  if (live && l < a.k) {
    a.idx[t * a.k + l] = sel;
    a.w[t * a.k + l] = w;
  }
}

// ---------------------------------------------------------------------------
// Gradient of the gate weights
// ---------------------------------------------------------------------------
// Slot l of a token: its expert (-1: none), scale * d_topk_w, and the expert's logit.
struct Slot {
  int id;
  float g, lg;
};
__device__ __forceinline__ Slot load_slot(const RouteBwdArgs& a, int64_t t, bool live, int l) {
  Slot s{-1, 0.f, -INFINITY};
  if (live && l < a.k) {
    s.id = a.idx[t * a.k + l];
    s.g = a.scale * a.d_w[t * a.k + l];
    if (s.id < 0 || s.id >= a.E) s.id = -1;
    if (s.id >= 0) {
      const float v = a.logits[t * a.E + s.id];
      s.lg = fminf(v, FLT_MAX);
      if (!(v > -INFINITY) || (a.bias && !(a.bias[s.id] > -INFINITY))) s.id = -1;  // not available: score 0
    }
  }
  return s;
}

// A slot's term of the gradient; the token's LT lanes together.  m, iz: largest logit and 1 / sum e^(l - m) of the
// row (plain softmax).
template <int LT>
__device__ __forceinline__ float slot_term(const RouteBwdArgs& a, const Slot& s, float m, float iz) {
  const bool has = s.id >= 0;
  if (a.renormalize) {
    float top = max_of<LT>(has ? s.lg : -FLT_MAX);
    if (a.sigmoid) top = fminf(top, 0.f);
    const float v = has ? scaled_score(a.sigmoid, s.lg, top) : 0.f, sum = sum_of<LT>(v);
    const float q = has ? v * inverse(sum) : 0.f;
    const float d = q * (s.g - sum_of<LT>(has ? q * s.g : 0.f));
    return a.sigmoid && has ? d * sigmoid_of(-s.lg) : d;  // 1 - s
  }
  if (!has) return 0.f;
  return a.sigmoid ? s.g * sigmoid_of(s.lg) * sigmoid_of(-s.lg) : s.g * (exp_of(s.lg - m) * iz);
}

// V consecutive logits from e, -inf where there are none or the expert is not available.
template <int V>
__device__ __forceinline__ void load_row(float (&x)[V], const float* row, const float* bias, int e, bool in) {
#pragma unroll
  for (int q = 0; q < V; ++q) x[q] = -INFINITY;
  if (in) {
    if constexpr (V == 4) {
      const floatx4 v = *reinterpret_cast<const floatx4*>(row + e);
#pragma unroll
      for (int q = 0; q < 4; ++q) x[q] = v[q];
    } else {
      x[0] = row[e];
    }
  }
#pragma unroll
  for (int q = 0; q < V; ++q) x[q] = x[q] > -INFINITY ? fminf(x[q], FLT_MAX) : -INFINITY;
  if (bias && in) {
#pragma unroll
    for (int q = 0; q < V; ++q)
      if (!(bias[e + q] > -INFINITY)) x[q] = -INFINITY;
  }
}
template <int V>
__device__ __forceinline__ void store_row(float* row, int e, const float (&o)[V]) {
  if constexpr (V == 4)
    __builtin_nontemporal_store(floatx4{o[0], o[1], o[2], o[3]}, reinterpret_cast<floatx4*>(row + e));
  else
    row[e] = o[0];
}

// HBM-bound: reads the chosen logits (the plain softmax's gradient: all of them), writes every gradient once.  TW
// tokens per wavefront: their slots side by side, 64 / TW lanes each, so that one chain of dependent loads (slot, then
// its logit) serves them all; then row by row over the whole wavefront, lane l holding V consecutive experts (4:
// 16-byte accesses, E % 4 == 0) from V (l + 64 i), i < PL.  The chosen experts' terms reach the lanes that hold them
// through a row of the wavefront's own in LDS, all slots at once: handed over one by one they cost 25 instructions a
// slot, 9.5 us at 16384 x 256 x 8 against 5.1.  A slot first leaves its number at its expert; one that finds
// another there shares its id, and then the wavefront's slots are added one after the other.
template <int TW, int V, int PL>
__global__ __launch_bounds__(kTokens* kWave) void route_rows_backward_kernel(RouteBwdArgs a) {
  extern __shared__ __attribute__((aligned(16))) float s_rows[];  // [kTokens][TW][Ep]
  constexpr int LT = 64 / TW, Ep = 64 * V * PL;
  const int lane = threadIdx.x & 63, sub = lane / LT;
  float* rows = s_rows + (threadIdx.x >> 6) * (TW * Ep);
  const int64_t t0 = ((int64_t)blockIdx.x * kTokens + (threadIdx.x >> 6)) * TW;
  const int E = a.E, k = a.k;
  const bool dense = !a.sigmoid && !a.renormalize;
  float o[TW][PL][V];
  if (dense)
#pragma unroll
    for (int w = 0; w < TW; ++w)
#pragma unroll
      for (int i = 0; i < PL; ++i) {
        const int e = V * (lane + 64 * i);
        load_row<V>(o[w][i], a.logits + (t0 + w) * E, a.bias, e, t0 + w < a.T && e < E);
      }
  const Slot s = load_slot(a, t0 + sub, t0 + sub < a.T, lane & (LT - 1));
  float m = 0.f, iz = 0.f;
  if (dense)
#pragma unroll
    for (int w = 0; w < TW; ++w) {
      float mw = -FLT_MAX, zw = 0.f;
#pragma unroll
      for (int i = 0; i < PL; ++i)
#pragma unroll
        for (int q = 0; q < V; ++q) mw = fmaxf(mw, o[w][i][q]);
      mw = max_of<64>(mw);
#pragma unroll
      for (int i = 0; i < PL; ++i)
#pragma unroll
        for (int q = 0; q < V; ++q) {
          o[w][i][q] = exp_of(o[w][i][q] - mw);
          zw += o[w][i][q];
        }
      zw = sum_of<64>(zw);
      zw = zw > 0.f ? inverse(zw) : 0.f;  // no expert is available: every term is zero
      m = sub == w ? mw : m;
      iz = sub == w ? zw : iz;
    }
  const float d = slot_term<LT>(a, s, m, iz);
  const float rest = dense ? -sum_of<LT>(d) * iz : 0.f;
  const bool has = s.id >= 0;
  float* at = rows + sub * Ep + (has ? s.id : 0);
  if (has) *at = __builtin_bit_cast(float, lane);
  wave_lds_order();
  const bool shared = __ballot(has && __builtin_bit_cast(int, *at) != lane) != 0;
  wave_lds_order();
#pragma unroll
  for (int w = 0; w < TW; ++w)
#pragma unroll
    for (int i = 0; i < PL; ++i)
#pragma unroll
      for (int q = 0; q < V; ++q) rows[w * Ep + V * (lane + 64 * i) + q] = 0.f;
  wave_lds_order();
  if (!shared) {
    if (has) *at = d;
  } else {
    for (int j = 0; j < k; ++j) {
      if (has && (lane & (LT - 1)) == j) *at += d;
      wave_lds_order();
    }
  }
  wave_lds_order();
#pragma unroll
  for (int w = 0; w < TW; ++w) {
    if (t0 + w >= a.T) break;  // wave-uniform
    const float rw = dense ? of_lane(rest, w * LT) : 0.f;
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      const int e = V * (lane + 64 * i);
      float v[V];
#pragma unroll
      for (int q = 0; q < V; ++q) v[q] = rows[w * Ep + e + q] + (dense ? o[w][i][q] * rw : 0.f);
      if (e < E) store_row<V>(a.d_logits + (t0 + w) * E, e, v);
    }
  }
}

// E <= 64, E % 4 == 0 and k <= 16: 16 lanes a token throughout, four experts a lane.
__global__ __launch_bounds__(kTokens* kWave) void route_small_backward_kernel(RouteBwdArgs a) {
  const int lane = threadIdx.x & 63, l = lane & 15, e = 4 * l;
  const int64_t t = ((int64_t)blockIdx.x * kTokens + (threadIdx.x >> 6)) * 4 + (lane >> 4);
  const bool live = t < a.T, in = live && e < a.E;
  const bool dense = !a.sigmoid && !a.renormalize;
  float o[4];
  load_row<4>(o, a.logits + t * a.E, a.bias, e, in && dense);
  const Slot s = load_slot(a, t, live, l);
  float m = 0.f, iz = 0.f;
  if (dense) {
    m = max_of<16>(fmaxf(fmaxf(fmaxf(o[0], o[1]), fmaxf(o[2], o[3])), -FLT_MAX));
    float z = 0.f;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      o[q] = exp_of(o[q] - m);
      z += o[q];
    }
    z = sum_of<16>(z);
    iz = z > 0.f ? inverse(z) : 0.f;
  }
  const float d = slot_term<16>(a, s, m, iz);
  const float rest = -sum_of<16>(d) * iz;
#pragma unroll
  for (int q = 0; q < 4; ++q) o[q] = dense ? o[q] * rest : 0.f;
  for (int j = 0; j < a.k; ++j) {
    const int id = __shfl(s.id, (lane & 48) + j);
    const float v = __shfl(d, (lane & 48) + j);
#pragma unroll
    for (int q = 0; q < 4; ++q) o[q] += e + q == id ? v : 0.f;
  }
  if (in) store_row<4>(a.d_logits + t * a.E, e, o);
}

}  // namespace

hipError_t launch_route_grouped(const RouteArgs& a, hipStream_t s) {
  const int n_group = a.topk_group < a.n_group ? a.n_group : 1;  // groups restrict the choice only if some are dropped
  const int Eg = a.E / n_group;
  auto bits_of = [&](int lt) {  // log2 of the lanes a group gets, or -1
    int bits = -1;
    while (n_group << (bits + 1) <= lt) ++bits;
    return bits;
  };
  auto per_lane = [&](int bits) { return bits < 0 ? 1 << 20 : (Eg + (1 << bits) - 1) >> bits; };
  const int b16 = bits_of(16), b64 = bits_of(64), p16 = per_lane(b16), p64 = per_lane(b64);  // p64 <= 32
  const bool vec4 = a.E % 4 == 0 && Eg % 4 == 0;
  // 16 lanes a token share the rounds of the selection between four tokens; 64 have fewer experts a lane to sort,
  // which is quicker until the tokens fill the chip (256 experts, 64 lanes against 16: 512 tokens 5.4 and 9.8 us,
  // 2048 9.1 and 9.9, 4096 10.8 and 10.0, 16384 24 and 16).
  const bool small = p16 <= 16 && a.k <= 16 && (p16 <= 4 || a.T > 2048);
  const int per_block = kTokens * (small ? 4 : 1);
  const dim3 grid((unsigned)((a.T + per_block - 1) / per_block)), block(kTokens * kWave);
  const Place pl{n_group, small ? b16 : b64, vec4};
#define MOE_ROUTE(LT_, PL_, PX_) hipLaunchKernelGGL((route_grouped_kernel<LT_, PL_, PX_>), grid, block, 0, s, a, pl, b64)
  if (small) {
    if (p16 <= 1) MOE_ROUTE(16, 1, 1);
    else if (p16 <= 2) MOE_ROUTE(16, 2, 1);
    else if (p16 <= 4) MOE_ROUTE(16, 4, 1);
    else if (p16 <= 8) MOE_ROUTE(16, 8, 2);
    else MOE_ROUTE(16, 16, 4);
  } else {
    if (p64 <= 1) MOE_ROUTE(64, 1, 1);
    else if (p64 <= 2) MOE_ROUTE(64, 2, 2);
    else if (p64 <= 4) MOE_ROUTE(64, 4, 4);
    else if (p64 <= 8) MOE_ROUTE(64, 8, 8);
    else if (p64 <= 16) MOE_ROUTE(64, 16, 16);
    else MOE_ROUTE(64, 32, 32);
  }
#undef MOE_ROUTE
  return hipGetLastError();
}

hipError_t launch_route_grouped_backward(const RouteBwdArgs& a, hipStream_t s) {
  const dim3 block(kTokens * kWave);
  const auto grid = [&](int per_wave) { return dim3((unsigned)((a.T + per_wave * kTokens - 1) / (per_wave * kTokens))); };
  // Four tokens a wavefront while their slots fit and the tokens fill the chip (256 experts, one against four: 512
  // tokens 2.9 and 3.3 us, 2048 3.0 and 3.1, 4096 3.6 and 3.4, 16384 6.0 and 4.4).
#define MOE_ROUTE(V_, PL_)                                                                                  \
  do {                                                                                                      \
    const size_t row = (size_t)kTokens * 64 * V_ * PL_ * sizeof(float);                                     \
    if (a.k <= 16 && a.T > 2048)                                                                            \
      hipLaunchKernelGGL((route_rows_backward_kernel<4, V_, PL_>), grid(4), block, 4 * row, s, a);          \
    else                                                                                                    \
      hipLaunchKernelGGL((route_rows_backward_kernel<1, V_, PL_>), grid(1), block, row, s, a);              \
  } while (0)
  if (a.E % 4 == 0) {
    if (a.E <= 64 && a.k <= 16) hipLaunchKernelGGL(route_small_backward_kernel, grid(4), block, 0, s, a);
    else if (a.E <= 256) MOE_ROUTE(4, 1);
    else if (a.E <= 512) MOE_ROUTE(4, 2);
    else MOE_ROUTE(4, 4);
  } else {
    if (a.E <= 64) MOE_ROUTE(1, 1);
    else if (a.E <= 256) MOE_ROUTE(1, 4);
    else MOE_ROUTE(1, 16);
  }
#undef MOE_ROUTE
  return hipGetLastError();
}

}  // namespace moe
