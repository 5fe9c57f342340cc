// A whole MoE layer for a few tokens (at most 64) in two launches (three with more than four tokens to route), over bf16
// or MXFP4 experts.
//
//   up    routes the tokens (or takes their experts), then a[t, e] = act(x_t W0_e (, x_t W0up_e)) * g(t, e)
//   down  out_t = sum over the token's local experts e of a[t, e] W1_e
//
// with g(t, e) the gate weight, summed over the token's slots that name e.  The layer is the reading of the chosen
// experts' weights: every weight is loaded once for four (or 16) of its expert's tokens, straight into the matrix
// instructions' registers, by as many wavefronts as it takes to keep HBM busy; nothing is permuted and no row is padded to
// a tile.  Measured: 4.5 TB/s of the chosen experts' weights with 64 tokens over 256 MXFP4 experts of 7168 x 2048 (1141
// us), 4.7 to 5.6 with 13 over 8 bf16 experts of 4096 x 2048 (58 to 70 us); 32 us for one token of 2048 x 1408, six
// experts, of which the dependent steps before the first weights are 4 to 5 us a launch.  Against routing, permute, grouped
// products and combine one after another, both captured (tile_m 16): 36 us and 61 for that token, 145 and 161 for one over
// bf16 experts of 7168 x 2048; but 259 and 227 for two of those, and 932 and 564 for 64 tokens over 8 bf16 experts of
// 4096 x 14336, whose weights are read again for each 16 tokens of an expert.
//
// v_mfma_f32_16x16x32_bf16 with 16 weight rows on its rows and tokens on its 16 columns: a column's result depends on
// its own token alone, so columns without a token hold anything.  MXFP4 weights are widened in registers to bf16, which
// is exact.  x is bf16; an activation goes between the launches in fp32 and enters the second product as three bf16
// terms (its upper eight bits of mantissa, the next eight, the last eight), so that the output keeps fp32 accuracy.
//
// Loading the tokens' side costs as many accesses as the weights' where every step of 32 reduction indices has its own
// load, most lanes of which have no token.  The narrow form gives an expert's tokens four at a time: one load has the
// four steps of a unit in its 16 columns, and a step's fragment is that register shifted by DPP.  The wide form, for
// more tokens an expert, has 16 at a time and a load a step.
#include "activation.h"

#include <type_traits>

namespace moe {
namespace {

constexpr uint32_t kOut = 0x80000000u;  // a byte offset past every resource
constexpr int kUnit = 128;              // reduction indices a wavefront loads at a time
constexpr int kUpWaves = 4, kDownWaves = 8;
constexpr int kTerms = 3;               // bf16 terms of an activation
constexpr int kNarrow = 4, kWide = 16;  // tokens of an expert at a time

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// What a workgroup knows about the routing, in LDS.  A token's choice of a local expert is a row of the activations:
// rows are ordered by expert, then token.  An entry is up to `batch` rows of one expert.
struct Lists {
  uint64_t* mask;     // [E_loc] tokens of each local expert
  int32_t* first;     // [E_loc] its first row
  uint32_t* entry;    // [entries] expert, rows << 16
  int32_t* row;       // [entries] first row
  int32_t* token;     // [rows] token of each row
  float* gate;        // [rows] its gate weight
  int32_t* idx;       // [T k]
  float* w;           // [T k]
  int n;              // entries
};

int max_entries(int T, int k, int E_loc, int batch) {
  const int rows = T * k, most = E_loc + rows / batch;
  return rows < most ? rows : most;
}
// (the device lays the arrays out for the smallest batches)
constexpr int kLeastBatch = kNarrow;
size_t lists_bytes(int T, int k, int E_loc) {
  return (size_t)E_loc * 12 + (size_t)(E_loc + T * k / kLeastBatch) * 8 + (size_t)T * k * 16 + 32;
}

// Reduction of a wavefront by DPP (rows of 16 lanes, then across them); every lane gets the result.
template <typename F>
__device__ __forceinline__ int wave_reduce(int v, int none, F f) {
  v = f(v, dpp<0x111>(none, v));       // row_shr:1, 2, 4, 8
  v = f(v, dpp<0x112>(none, v));
  v = f(v, dpp<0x114>(none, v));
  v = f(v, dpp<0x118>(none, v));
  v = f(v, dpp<0x142, 0xa>(none, v));  // row_bcast:15 into rows 1 and 3
  v = f(v, dpp<0x143, 0xc>(none, v));  // row_bcast:31 into rows 2 and 3
  return __builtin_amdgcn_readlane(v, 63);
}
// Sums of lanes 0 .. l.
__device__ __forceinline__ int wave_scan(int v) {
  v += dpp<0x111>(0, v);
  v += dpp<0x112>(0, v);
  v += dpp<0x114>(0, v);
  v += dpp<0x118>(0, v);
  v += dpp<0x142, 0xa>(0, v);
  v += dpp<0x143, 0xc>(0, v);
  return v;
}
// A float's order as an int's.
__device__ __forceinline__ int ordered(float f) {
  const int b = __builtin_bit_cast(int, f);
  return b ^ ((b >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float from_ordered(int b) { return __builtin_bit_cast(float, b ^ ((b >> 31) & 0x7fffffff)); }

// Top-k of one row by one wavefront, as moe_route_topk does it: lane l holds logits l, l + 64, ...  Experts whose logit
// is -inf or NaN are never chosen and have no part in a softmax's sum; +inf counts as the largest number.
__device__ __forceinline__ void route_row(const float* row, int E, int k, bool renormalize, int32_t* idx, float* w) {
  constexpr int PL = 16;
  constexpr int kNone = (int)0x80000000;  // below every number's key
  const int lane = threadIdx.x & 63, per = (E + 63) / 64;
  int v[PL];
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    if (i >= per) break;
    const int e = lane + i * 64;
    const float l = e < E ? row[e] : -__builtin_inff();
    // (-0 and 0 are equal: adding 0 makes them the same)
    v[i] = l > -__builtin_inff() ? ordered(fminf(l, 3.402823466e38f) + 0.0f) : kNone;
  }
  float top = 0.f, sum = 0.f, mine_v = 0.f, all = 0.f;
  int mine = -1;
  for (int j = 0; j < k; ++j) {
    int best = kNone, id = 0;
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      if (i >= per) break;
      if (v[i] > best) {
        best = v[i];
        id = lane + i * 64;
      }
    }
    const int m = wave_reduce(best, kNone, [](int a, int b) { return a > b ? a : b; });
    if (m == kNone) break;  // none left: this slot and those after it stay empty
    const float l = from_ordered(m);
    if (j == 0) {
      top = l;
      if (!renormalize) {
#pragma unroll
        for (int i = 0; i < PL; ++i) {
          if (i >= per) break;
          if (v[i] != kNone) all += expf(from_ordered(v[i]) - top);
        }
      }
    }
    // Equal logits: the lowest id.
    const uint64_t holds = __ballot(best == m);
    int b;
    if ((holds & (holds - 1)) == 0) b = __builtin_amdgcn_readlane(id, __builtin_ctzll(holds));
    else b = wave_reduce(best == m ? id : 0x7fffffff, 0x7fffffff, [](int a, int c) { return a < c ? a : c; });
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      if (i >= per) break;
      if (b == lane + i * 64) v[i] = kNone;
    }
    const float z = expf(l - top);
    sum += z;
    if (lane == j) {
      mine = b;
      mine_v = z;
    }
  }
  if (!renormalize) {
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) all += __shfl_xor(all, o);
    sum = all;
  }
  if (lane < k) {
    idx[lane] = mine;
    w[lane] = mine >= 0 ? mine_v / sum : 0.f;
  }
}

// A wavefront a token: the latency of its loads and of k searches one after another.
__global__ __launch_bounds__(64) void route_kernel(FewArgs a) {
  const int t = blockIdx.x;
  route_row(a.logits + (int64_t)t * a.E, a.E, a.k, a.renormalize, a.topk_idx + t * a.k, a.topk_w + t * a.k);
}

// Fills the lists; the whole workgroup takes part.  out: the workgroup that hands the routing's results out.
template <int THREADS, int BATCH>
__device__ __forceinline__ Lists make_lists(const FewArgs& a, const float* logits, char* smem, bool out) {
  const int pairs = a.T * a.k, entries = a.E_loc + pairs / kLeastBatch;
  Lists l;
  l.mask = reinterpret_cast<uint64_t*>(smem);
  l.first = reinterpret_cast<int32_t*>(l.mask + a.E_loc);
  l.entry = reinterpret_cast<uint32_t*>(l.first + a.E_loc);
  l.row = reinterpret_cast<int32_t*>(l.entry + entries);
  l.token = l.row + entries;
  l.gate = reinterpret_cast<float*>(l.token + pairs);
  l.idx = reinterpret_cast<int32_t*>(l.gate + pairs);
  l.w = reinterpret_cast<float*>(l.idx + pairs);
  int32_t* total = reinterpret_cast<int32_t*>(l.w + pairs);
  int32_t* twice = total + 1;  // some token's choice names an expert twice
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  // One token: a lane a slot of one wavefront, entries in slot order, without the steps between workgroup barriers (56.6 us
  // instead of 59.2 for 8 of 256 MXFP4 experts of 7168 x 2048).
  if (a.T == 1) {
    if (wave == 0) {
      if (logits) route_row(logits, a.E, a.k, a.renormalize, l.idx, l.w);
      const int id = lane >= a.k ? -1 : logits ? l.idx[lane] : a.topk_idx[lane];
      const float own = lane >= a.k ? 0.f : logits ? l.w[lane] : a.topk_w[lane];
      const uint32_t e = (uint32_t)id - (uint32_t)a.expert_begin;
      bool first = id >= 0 && e < (uint32_t)a.E_loc;
      float w = own;
      for (int q = 0; q < a.k; ++q) {  // (a choice that names an expert twice has both weights in one row)
        const bool same = __builtin_amdgcn_readlane(id, q) == id;
        first = first && !(same && q < lane);
        if (same && q > lane) w += __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, own), q));
      }
      const uint64_t firsts = __ballot(first);
      if (first) {
        const int r = __popcll(firsts & ((1ull << lane) - 1));
        l.entry[r] = e | 1u << 16;
        l.row[r] = r;
        l.token[r] = 0;
        l.gate[r] = w;
      }
      if (lane == 0) *total = __popcll(firsts);
      if (logits && out && lane < a.k) {
        a.topk_idx[lane] = id;
        a.topk_w[lane] = own;
      }
    }
    __syncthreads();
    l.n = *total;
    return l;
  }
  for (int e = tid; e < a.E_loc; e += THREADS) l.mask[e] = 0;
  if (tid == 0) *twice = 0;
  if (logits) {
    for (int t = wave; t < a.T; t += THREADS / 64)
      route_row(logits + (int64_t)t * a.E, a.E, a.k, a.renormalize, l.idx + t * a.k, l.w + t * a.k);
  } else {
    for (int p = tid; p < pairs; p += THREADS) {
      l.idx[p] = a.topk_idx[p];
      l.w[p] = a.topk_w[p];
    }
  }
  __syncthreads();
  for (int p = tid; p < pairs; p += THREADS) {
    const int32_t id = l.idx[p];
    const uint32_t e = (uint32_t)id - (uint32_t)a.expert_begin;
    if (id >= 0 && e < (uint32_t)a.E_loc) {
      const unsigned long long bit = 1ull << (p / a.k);
      if (atomicOr(reinterpret_cast<unsigned long long*>(l.mask + e), bit) & bit) *twice = 1;
    }
    if (logits && out) {
      a.topk_idx[p] = id;
      a.topk_w[p] = l.w[p];
    }
  }
  __syncthreads();
  if (wave == 0) {
    int n = 0, rows = 0;
    for (int e0 = 0; e0 < a.E_loc; e0 += 64) {
      const int e = e0 + lane;
      const int own = e < a.E_loc ? __popcll(l.mask[e]) : 0, parts = (own + BATCH - 1) / BATCH;
      const int c = wave_scan(own | parts << 16);  // running sums of both (rows <= 2048)
      const int r0 = rows + (c & 0xffff) - own, n0 = n + (c >> 16) - parts;
      if (e < a.E_loc) l.first[e] = r0;
      for (int i = 0; i < parts; ++i) {
        const int left = own - i * BATCH;
        l.entry[n0 + i] = (uint32_t)e | (uint32_t)(left < BATCH ? left : BATCH) << 16;
        l.row[n0 + i] = r0 + i * BATCH;
      }
      const int last = __builtin_amdgcn_readlane(c, 63);
      rows += last & 0xffff;
      n += last >> 16;
    }
    if (lane == 0) *total = n;
  }
  __syncthreads();
  // Each row's token and gate weight.  (A choice that names an expert twice has both weights in one row.)
  const bool repeats = *twice != 0;
  for (int p = tid; p < pairs; p += THREADS) {
    const int32_t id = l.idx[p];
    const uint32_t e = (uint32_t)id - (uint32_t)a.expert_begin;
    if (id < 0 || e >= (uint32_t)a.E_loc) continue;
    const int t = p / a.k, end = (t + 1) * a.k;
    float w = l.w[p];
    if (repeats) {
      bool again = false;
      for (int q = t * a.k; q < p; ++q) again |= l.idx[q] == id;
      if (again) continue;
      for (int q = p + 1; q < end; ++q) w += l.idx[q] == id ? l.w[q] : 0.f;
    }
    const int r = l.first[e] + __popcll(l.mask[e] & ((1ull << t) - 1));
    l.token[r] = t;
    l.gate[r] = w;
  }
  __syncthreads();
  l.n = *total;
  return l;
}

// A unit of 16 weight rows: 128 reduction indices a row, as a lane holds them.  (Loads of 64 bytes a row, half a cache
// line, that are not marked as streaming: the next unit's take the other half from the cache.  Marked, the bf16 layer
// of 32 experts of 7168 x 2048 took 597 us instead of 524.)
template <bool FP4>
struct Weights;
template <>
struct Weights<false> {  // step s: indices 32 s + 8 (lane / 16) + 0..7 of row lane % 16
  u32x4 v[4];
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t row, int K, int unit, bool in) {
    const int g = (threadIdx.x >> 4) & 3;
    const uint32_t at = row * (uint32_t)(K * 2) + unit * 256 + g * 16;
#pragma unroll
    for (int s = 0; s < 4; ++s) v[s] = __builtin_amdgcn_raw_buffer_load_b128(r, in ? at + s * 64 : kOut, 0, 0);
  }
  __device__ __forceinline__ bf16x8 get(int s, uint32_t) const { return __builtin_bit_cast(bf16x8, v[s]); }
  static __device__ __forceinline__ uint32_t token_at(int unit, int s) { return unit * 256 + s * 64 + ((threadIdx.x >> 4) & 3) * 16; }
};
template <>
struct Weights<true> {  // step s: indices 32 (lane / 16) + 8 s + 0..7 of row lane % 16: a lane has one block
  u32x4 v;
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t row, int K, int unit, bool in) {
    const int g = (threadIdx.x >> 4) & 3;
    v = __builtin_amdgcn_raw_buffer_load_b128(r, in ? row * (uint32_t)(K / 2) + unit * 64 + g * 16 : kOut, 0, 0);
  }
  // scales: the unit's four scale bytes of the row
  __device__ __forceinline__ bf16x8 get(int s, uint32_t scales) const {
    const float scale = mxfp4_scale((scales >> (8 * ((threadIdx.x >> 4) & 3))) & 255u);
    struct { bf16x2 p[4]; } o;
    o.p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v[s], scale, 0);
    o.p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v[s], scale, 1);
    o.p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v[s], scale, 2);
    o.p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v[s], scale, 3);
    return __builtin_bit_cast(bf16x8, o);
  }
  static __device__ __forceinline__ uint32_t token_at(int unit, int s) { return unit * 256 + ((threadIdx.x >> 4) & 3) * 64 + s * 16; }
};

template <bool FP4>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t codes_rsrc(const void* w, int64_t row0, int rows, int K) {
  const int64_t b = FP4 ? K / 2 : K * 2;
  return make_rsrc(static_cast<const char*>(w) + row0 * b, rows * b);
}

// Units go in groups of four, whose scales, 16 bytes a row, come as one load: a load of four bytes a row for each unit
// cost as many cache accesses as the codes (431 us instead of 310 without any for 64 experts of 7168 x 2048).
constexpr int kGroup = 4;

template <bool FP4, int M>
struct GroupScales {
  u32x4 v[M];
};
template <int M>
struct GroupScales<false, M> {};

// Calls f with the steps 0..3 as constants.
template <typename F>
__device__ __forceinline__ void each_step(F f) {
  f(std::integral_constant<int, 0>{});
  f(std::integral_constant<int, 1>{});
  f(std::integral_constant<int, 2>{});
  f(std::integral_constant<int, 3>{});
}

// ---------------------------------------------------------------------------
// First launch
// ---------------------------------------------------------------------------
// An item is an entry's 16 R rows of the gate (and up) matrix; a workgroup's wavefronts take turns at groups of its
// reduction's units and add up through LDS.
// Rows: fewer leave enough items for the CUs, more share a load of the tokens.
constexpr int up_rows(bool fp4, bool wide) { return fp4 && wide ? 4 : fp4 || wide ? 2 : 1; }
// Workgroups a CU holds: as many as leave the registers that the loads in flight need.
constexpr int up_per_cu(bool fp4, int nmat, bool wide) { return nmat == 2 && (wide || fp4) ? (wide ? 2 : 3) : 4 - wide; }

template <bool FP4, int NMAT, bool WIDE>
__global__ __launch_bounds__(kUpWaves * 64, up_per_cu(FP4, NMAT, WIDE)) void up_kernel(FewArgs a, bool zero) {
  constexpr int R = up_rows(FP4, WIDE), MR = NMAT * R, D = 2, XL = WIDE ? 4 : 1;
  constexpr int RED = MR * 256, STEP = kUpWaves * kGroup;
  extern __shared__ __attribute__((aligned(16))) char smem[];
  float* red = reinterpret_cast<float*>(smem);
  if (zero)  // the second launch adds to out
    for (int i = blockIdx.x * (kUpWaves * 64) + threadIdx.x; i < a.T * a.H / 4; i += gridDim.x * (kUpWaves * 64))
      reinterpret_cast<floatx4*>(a.out)[i] = floatx4{0.f, 0.f, 0.f, 0.f};
  const Lists l = make_lists<kUpWaves * 64, WIDE ? kWide : kNarrow>(a, a.logits, smem + kUpWaves * RED * 4, blockIdx.x == 0);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, g = lane >> 4, column = WIDE ? l16 : l16 & 3;
  const int blocks = a.F / (16 * R), items = l.n * blocks, units = a.H / kUnit;
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(a.x, (int64_t)a.T * a.H * 2);
  float* activations = static_cast<float*>(a.ws);
  const void* wp[2] = {a.w0, a.w0_up};
  const uint8_t* sp[2] = {a.s0, a.s0_up};

  for (int item = blockIdx.x; item < items; item += gridDim.x) {
    const int at = item / blocks, f0 = (item - at * blocks) * 16 * R;
    const uint32_t entry = (uint32_t)__builtin_amdgcn_readfirstlane((int)l.entry[at]);
    const int e = entry & 0xffff, n = entry >> 16, first = __builtin_amdgcn_readfirstlane(l.row[at]);
    const uint32_t xo = column < n ? (uint32_t)(l.token[first + column] * a.H * 2) : kOut;
    const int64_t row0 = (int64_t)e * a.F + f0;
    __amdgpu_buffer_rsrc_t rw[NMAT], rs[NMAT];
#pragma unroll
    for (int m = 0; m < NMAT; ++m) {
      rw[m] = codes_rsrc<FP4>(wp[m], row0, 16 * R, a.H);
      rs[m] = FP4 ? make_rsrc(sp[m] + row0 * (a.H / 32), 16 * R * (a.H / 32)) : rw[m];
    }
    floatx4 acc[MR];
#pragma unroll
    for (int m = 0; m < MR; ++m) acc[m] = floatx4{0.f, 0.f, 0.f, 0.f};
    Weights<FP4> w[D][MR];
    u32x4 x[D][XL];
    auto load = [&](int q, int u) {
      const bool in = u < units;
#pragma unroll
      for (int m = 0; m < MR; ++m) w[q][m].load(rw[m / R], (m % R) * 16 + l16, a.H, u, in);
#pragma unroll
      for (int s = 0; s < XL; ++s)
        x[q][s] = __builtin_amdgcn_raw_buffer_load_b128(rx, in ? xo + Weights<FP4>::token_at(u, WIDE ? s : l16 >> 2) : kOut, 0, 0);
    };
    GroupScales<FP4, MR> sc, next;
    auto load_scales = [&](GroupScales<FP4, MR>& v, int u) {  // (may run into the next row's, which no unit uses)
      if constexpr (FP4)
#pragma unroll
        for (int m = 0; m < MR; ++m)
          v.v[m] = __builtin_amdgcn_raw_buffer_load_b128(
              rs[m / R], u < units ? (uint32_t)(((m % R) * 16 + l16) * (a.H / 32) + u * 4) : kOut, 0, 0);
    };
    load_scales(next, wave * kGroup);
#pragma unroll
    for (int q = 0; q < D; ++q) load(q, wave * kGroup + q);
    for (int u = wave * kGroup; u < units; u += STEP) {
      sc = next;
      load_scales(next, u + STEP);
#pragma unroll
      for (int j = 0; j < kGroup; ++j) {
        each_step([&](auto step) {
          constexpr int S = decltype(step)::value;
          const bf16x8 t = __builtin_bit_cast(bf16x8, WIDE ? x[j % D][WIDE ? S : 0] : shifted<WIDE ? 0 : 4 * S>(x[j % D][0]));
#pragma unroll
          for (int m = 0; m < MR; ++m) {
            uint32_t scales = 0;  // (past the row's end the codes are zeros, and so is their scale)
            if constexpr (FP4) scales = u + j < units ? sc.v[m][j] : 0;
            acc[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[j % D][m].get(S, scales), t, acc[m], 0, 0, 0);
          }
        });
        load(j % D, j + D < kGroup ? u + j + D : u + STEP + j + D - kGroup);
      }
    }
    __syncthreads();  // (the last item's sums have been read)
#pragma unroll
    for (int m = 0; m < MR; ++m) *reinterpret_cast<floatx4*>(red + wave * RED + m * 256 + lane * 4) = acc[m];
    __syncthreads();
    // Lane: the entry's row l16, weight rows 4 g + 0..3 of a block of 16.
    for (int r = wave; r < R; r += kUpWaves) {
      floatx4 z = {0.f, 0.f, 0.f, 0.f}, u = z;
#pragma unroll
      for (int v = 0; v < kUpWaves; ++v) {
        z += *reinterpret_cast<const floatx4*>(red + v * RED + r * 256 + lane * 4);
        if (NMAT == 2) u += *reinterpret_cast<const floatx4*>(red + v * RED + (R + r) * 256 + lane * 4);
      }
      if (l16 < n) {
        const float gate = l.gate[first + l16];
        floatx4 y;
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = (NMAT == 2 ? activate(ACT_SILU, z[i]) * u[i] : activate(ACT_GELU, z[i])) * gate;
        *reinterpret_cast<floatx4*>(activations + (int64_t)(first + l16) * a.F + f0 + r * 16 + g * 4) = y;
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Second launch
// ---------------------------------------------------------------------------
// Eight activations as three bf16 terms whose sum they are, each of the activation's sign.  The first is zero, infinite or
// NaN where the activation is; what the others are then does not count (with_rest).
struct Terms {
  u32x4 t[kTerms];
};
__device__ __forceinline__ Terms split(floatx4 lo, floatx4 hi) {
  Terms o;
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    float a[2] = {i < 4 ? lo[i & 3] : hi[i & 3], i < 4 ? lo[(i & 3) + 1] : hi[(i & 3) + 1]};
#pragma unroll
    for (int c = 0; c < kTerms; ++c) {
      const uint32_t b0 = __builtin_bit_cast(uint32_t, a[0]), b1 = __builtin_bit_cast(uint32_t, a[1]);
      o.t[c][i >> 1] = __builtin_amdgcn_perm(b1, b0, 0x07060302u);  // the upper halves
#pragma unroll
      for (int e = 0; e < 2; ++e) a[e] -= __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, a[e]) & 0xffff0000u);
    }
  }
  return o;
}

// Sums of the first terms' products and of the others'.  Where the first terms' is an infinity or NaN it is the result: an
// infinite weight, or activation, makes NaN of a later term that is zero (an activation of few bits), or of inf - inf.
__device__ __forceinline__ floatx4 with_rest(floatx4 first, floatx4 rest) {
  floatx4 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = fabsf(first[i]) < __builtin_inff() ? rest[i] + first[i] : first[i];
  return o;
}

// The narrow form's fragment of step S: columns 4 c + p are term c of row p, from columns 4 S + p.
template <int S, int C>
__device__ __forceinline__ void place_term(u32x4& o, u32x4 t) {
  constexpr int by = 4 * (S - C), ctrl = by == 0 ? 0xE4 : by > 0 ? 0x100 + by : 0x110 - by;  // quad_perm 0123, row_shl, row_shr
#pragma unroll
  for (int i = 0; i < 4; ++i)
    o[i] = (uint32_t)__builtin_amdgcn_update_dpp((int)o[i], (int)t[i], ctrl, 0xf, 1 << C, false);
}

// A workgroup has 16 R output columns of every token, of all units or (S = 2) of half of them; its wavefronts take turns
// at the entries' groups of units, and each adds each group's sums to the tokens' in LDS, a copy for each wavefront, so
// that the order of additions is fixed.  With S = 2 the two workgroups add to out, which the first launch has cleared:
// two terms make the same sum in either order.
template <bool FP4, bool WIDE, int R>
__global__ __launch_bounds__(kDownWaves * 64, WIDE || R == 4 ? 2 : 4) void down_kernel(FewArgs a, int S) {
  constexpr int D = 2, G = kGroup, PITCH = 16 * R + 4, XL = WIDE ? 4 : 1;
  extern __shared__ __attribute__((aligned(16))) char smem[];
  float* sums = reinterpret_cast<float*>(smem);  // [wavefront][token][PITCH]
  const int each = a.T * PITCH;
  for (int i = threadIdx.x; i < kDownWaves * each / 4; i += kDownWaves * 64)
    reinterpret_cast<floatx4*>(sums)[i] = floatx4{0.f, 0.f, 0.f, 0.f};
  const Lists l = make_lists<kDownWaves * 64, WIDE ? kWide : kNarrow>(a, nullptr, smem + kDownWaves * each * 4, false);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, g = lane >> 4, column = WIDE ? l16 : l16 & 3;
  const int h0 = (int)(blockIdx.x / S) * 16 * R, per = a.F / kUnit, pg = (per + G - 1) / G;
  const int part = (int)(blockIdx.x % S), g0 = (int)((int64_t)part * l.n * pg / S), g1 = (int)((int64_t)(part + 1) * l.n * pg / S);
  const float* activations = static_cast<const float*>(a.ws);
  float* mine = sums + wave * each;

  struct Group {
    __amdgpu_buffer_rsrc_t rw, rs, rt;
    uint32_t off;  // of this lane's activation row
    int unit, n, first;
  };
  auto group = [&](int i) {
    Group v;
    const bool in = i < g1;
    const int at = in ? i / pg : 0;
    const uint32_t entry = in ? (uint32_t)__builtin_amdgcn_readfirstlane((int)l.entry[at]) : 0;
    const int e = entry & 0xffff;
    v.n = entry >> 16;
    v.first = in ? __builtin_amdgcn_readfirstlane(l.row[at]) : 0;
    v.unit = in ? (i - at * pg) * G : per;  // (units from `per` on load from past the resources)
    const int64_t row0 = (int64_t)e * a.H + h0;
    v.rw = codes_rsrc<FP4>(a.w1, row0, 16 * R, a.F);
    v.rs = FP4 ? make_rsrc(a.s1 + row0 * (a.F / 32), 16 * R * (a.F / 32)) : v.rw;
    v.rt = make_rsrc(activations + (int64_t)v.first * a.F, (int64_t)v.n * a.F * 4);
    v.off = column < v.n ? (uint32_t)(column * a.F * 4) : kOut;
    return v;
  };
  Weights<FP4> w[D][R];
  floatx4 x[D][XL][2];
  auto load = [&](int q, const Group& v, int j) {  // the group's j-th unit
    const int u = v.unit + j;
    const bool in = u < per;
#pragma unroll
    for (int r = 0; r < R; ++r) w[q][r].load(v.rw, r * 16 + l16, a.F, u, in);
#pragma unroll
    for (int s = 0; s < XL; ++s)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        x[q][s][h] = __builtin_bit_cast(floatx4, __builtin_amdgcn_raw_buffer_load_b128(
                         v.rt, in ? v.off + 2 * Weights<FP4>::token_at(u, WIDE ? s : l16 >> 2) + 16 * h : kOut, 0, 0));
  };
  auto load_scales = [&](GroupScales<FP4, R>& s, const Group& v) {
    if constexpr (FP4)
#pragma unroll
      for (int r = 0; r < R; ++r)
        s.v[r] = __builtin_amdgcn_raw_buffer_load_b128(
            v.rs, v.unit < per ? (uint32_t)((r * 16 + l16) * (a.F / 32) + v.unit * 4) : kOut, 0, 0);
  };
  GroupScales<FP4, R> sc, next;
  Group cur = group(g0 + wave);
  load_scales(next, cur);
#pragma unroll
  for (int q = 0; q < D; ++q) load(q, cur, q);
  for (int i = g0 + wave; i < g1; i += kDownWaves) {
    const Group ahead = group(i + kDownWaves);
    sc = next;
    load_scales(next, ahead);
    floatx4 acc[R], rest[WIDE ? R : 1];  // wide: the first terms' sums, the others' (narrow: columns of one)
#pragma unroll
    for (int r = 0; r < R; ++r) {
      acc[r] = floatx4{0.f, 0.f, 0.f, 0.f};
      if constexpr (WIDE) rest[r] = acc[r];
    }
#pragma unroll
    for (int j = 0; j < G; ++j) {
      Terms t;
      if constexpr (!WIDE) t = split(x[j % D][0][0], x[j % D][0][1]);
      each_step([&](auto step) {
        constexpr int T = decltype(step)::value;
        if constexpr (WIDE) {
          t = split(x[j % D][T][0], x[j % D][T][1]);
        }
        u32x4 b = {0, 0, 0, 0};
        if constexpr (!WIDE) {
          place_term<T, 0>(b, t.t[0]);
          place_term<T, 1>(b, t.t[1]);
          place_term<T, 2>(b, t.t[2]);
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
          uint32_t scales = 0;
          if constexpr (FP4) scales = cur.unit + j < per ? sc.v[r][j] : 0;
          const bf16x8 f = w[j % D][r].get(T, scales);
          if constexpr (WIDE) {
#pragma unroll
            for (int c = 0; c < kTerms; ++c) {
              floatx4& to = c == 0 ? acc[r] : rest[r];
              to = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f, __builtin_bit_cast(bf16x8, t.t[c]), to, 0, 0, 0);
            }
          } else {
            acc[r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f, __builtin_bit_cast(bf16x8, b), acc[r], 0, 0, 0);
          }
        }
      });
      if (j + D < G) load(j % D, cur, j + D);
      else load(j % D, ahead, j + D - G);
    }
    const int token = l16 < cur.n ? l.token[cur.first + l16] : 0;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      floatx4 t;
      if constexpr (WIDE) {
        t = with_rest(acc[r], rest[r]);
      } else {  // the terms' columns, smallest first
        const u32x4 bits = __builtin_bit_cast(u32x4, acc[r]);
        t = with_rest(acc[r], __builtin_bit_cast(floatx4, shifted<8>(bits)) + __builtin_bit_cast(floatx4, shifted<4>(bits)));
      }
      if (l16 < cur.n) *reinterpret_cast<floatx4*>(mine + token * PITCH + r * 16 + g * 4) += t;
    }
    cur = ahead;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < a.T * 4 * R; i += kDownWaves * 64) {
    const int t = i / (4 * R), c = (i - t * 4 * R) * 4;
    floatx4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int v = 0; v < kDownWaves; ++v) o += *reinterpret_cast<const floatx4*>(sums + v * each + t * PITCH + c);
    float* to = a.out + (int64_t)t * a.H + h0 + c;
    if (S == 1) {
      *reinterpret_cast<floatx4*>(to) = o;
    } else {
#pragma unroll
      for (int v = 0; v < 4; ++v) unsafeAtomicAdd(to + v, o[v]);
    }
  }
}

constexpr size_t kLds = 160 << 10;  // of a workgroup
size_t down_sums(int T, int R) { return (size_t)kDownWaves * T * (16 * R + 4) * 4; }

int cu_count() {
  int dev = 0, n = 0;
  if (hipGetDevice(&dev) != hipSuccess || hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess)
    return 256;
  return n;
}

template <bool FP4, int NMAT, bool WIDE, int R2>
hipError_t launch_both(const FewArgs& a, hipStream_t s) {
  constexpr int R = up_rows(FP4, WIDE);
  const size_t lists = lists_bytes(a.T, a.k, a.E_loc);
  const int cus = cu_count();
  // Too few column blocks for two workgroups a CU: half of the reduction each.
  const int columns = a.H / (16 * R2), S = columns < 2 * cus ? 2 : 1;
  const int64_t items = (int64_t)max_entries(a.T, a.k, a.E_loc, WIDE ? kWide : kNarrow) * (a.F / (16 * R));
  const int64_t most = (int64_t)cus * up_per_cu(FP4, NMAT, WIDE);
  hipLaunchKernelGGL((up_kernel<FP4, NMAT, WIDE>), dim3((unsigned)(items < most ? items : most)), dim3(kUpWaves * 64),
                     (size_t)kUpWaves * NMAT * R * 1024 + lists, s, a, S == 2);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((down_kernel<FP4, WIDE, R2>), dim3((unsigned)(columns * S)), dim3(kDownWaves * 64),
                     down_sums(a.T, R2) + lists, s, a, S);
  return hipGetLastError();
}

template <bool FP4, bool WIDE>
hipError_t launch(const FewArgs& a, hipStream_t s) {
  const auto with = [&](auto rows) {
    constexpr int R = decltype(rows)::value;
    return a.w0_up ? launch_both<FP4, 2, WIDE, R>(a, s) : launch_both<FP4, 1, WIDE, R>(a, s);
  };
  if constexpr (FP4) {
    // The most rows (fewer loads of the activations) that leave three CUs in four a workgroup, each half of a block's
    // reduction: four instead of two for out of 7168 1139 us, 1203 (64 tokens, 256 experts of 2048), but of 4096 422 us, 353
    // (32 tokens, 128 experts of 2048); one instead of two for out of 2048 78 us, 88 (16 tokens, 64 experts of 1408).
    const auto enough = [&](int R) { return 2 * (a.H / (16 * R)) >= cu_count() / 4 * 3; };
    if constexpr (!WIDE)
      if (enough(4) && down_sums(a.T, 4) + lists_bytes(a.T, a.k, a.E_loc) <= kLds) return with(std::integral_constant<int, 4>{});
    if (enough(2)) return with(std::integral_constant<int, 2>{});
  }
  return with(std::integral_constant<int, 1>{});
}

}  // namespace

size_t few_tokens_ws_bytes(int T, int k, int F) { return (size_t)T * k * F * 4; }

hipError_t launch_few_tokens(const FewArgs& args, hipStream_t s) {
  FewArgs a = args;
  // Every workgroup of the first launch routes for itself, a wavefront a token, if each has one token at most (four tokens
  // of 2048 x 1408 over 64 experts 76.0 us, 77.7 with a launch for it).  More are routed by a launch of their own, 8 us
  // (64 tokens of 7168 x 2048 over 256 experts 1141 us, 1236 without it; 5 tokens of 2048 x 1408 88.3, 89.3).
  if (a.logits && a.T > kUpWaves) {
    hipLaunchKernelGGL(route_kernel, dim3((unsigned)a.T), dim3(64), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    a.logits = nullptr;
  }
  // The wide form where experts have more than three tokens on average.
  const bool wide = a.T > kNarrow && a.T * a.k > 3 * a.E;
  if (a.s0) return wide ? launch<true, true>(a, s) : launch<true, false>(a, s);
  return wide ? launch<false, true>(a, s) : launch<false, false>(a, s);
}

}  // namespace moe
