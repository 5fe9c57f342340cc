// A whole MoE layer for a few tokens (at most 64) in two launches, over bf16 or MXFP4 experts.
//
//   up    routes the tokens (or takes their experts), then a[t, e] = act(x_t W0_e (, x_t W0up_e)) * g(t, e)
//   down  out_t = sum over the token's local experts e of a[t, e] W1_e
//
// with g(t, e) the gate weight, summed over the token's slots that name e.  The layer is the reading of the chosen
// experts' weights: every weight is loaded once, straight into the matrix instructions' registers, by as many
// wavefronts as it takes to keep HBM busy; nothing is permuted and no row is padded to a tile.
//
// v_mfma_f32_16x16x32_bf16 with 16 weight rows on its rows and up to 16 tokens on its columns: a column's result
// depends on its own token alone, so columns without a token hold anything.  MXFP4 weights are widened in registers to
// bf16, which is exact.  x is bf16; the activations go between the launches as two bf16 terms (a value and the
// remainder, 16 bits of mantissa), so that the output keeps fp32 accuracy: the second product costs twice the matrix
// instructions, which the loads hide.
#include "activation.h"

namespace moe {
namespace {

constexpr uint32_t kOut = 0x80000000u;  // a byte offset past every resource
constexpr int kUnit = 128;              // reduction indices a wavefront loads at a time
constexpr int kUpWaves = 4, kDownWaves = 8;

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
// (the device lays the arrays out for batches of 16, the smallest)
size_t lists_bytes(int T, int k, int E_loc) {
  return (size_t)E_loc * 12 + (size_t)(E_loc + T * k / 16) * 8 + (size_t)T * k * 16 + 32;
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor(v, o));
  return v;
}

// Top-k of one row by one wavefront, as moe_route_topk does it: lane l holds logits l, l + 64, ...  Experts whose logit
// is -inf or NaN are never chosen and have no part in a softmax's sum; +inf counts as the largest number.
__device__ __forceinline__ void route_row(const float* row, int E, int k, bool renormalize, int32_t* idx, float* w) {
  constexpr int PL = 16;
  const int lane = threadIdx.x & 63, per = (E + 63) / 64;
  const float ninf = -__builtin_inff();
  float v[PL];
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    if (i >= per) break;
    const int e = lane + i * 64;
    const float l = e < E ? row[e] : ninf;
    v[i] = l > ninf ? fminf(l, 3.402823466e38f) : ninf;
  }
  float top = 0.f, sum = 0.f, mine_v = 0.f, all = 0.f;
  int mine = -1;
  for (int j = 0; j < k; ++j) {
    float best = ninf;
    int id = 0x7fffffff;
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      if (i >= per) break;
      if (v[i] > best) {
        best = v[i];
        id = lane + i * 64;
      }
    }
    const float m = wave_max(best);
    if (!(m > ninf)) break;  // none left: this slot and those after it stay empty
    if (j == 0) {
      top = m;
      if (!renormalize) {
#pragma unroll
        for (int i = 0; i < PL; ++i) {
          if (i >= per) break;
          if (v[i] > ninf) all += expf(v[i] - top);
        }
      }
    }
    int b = best == m ? id : 0x7fffffff;
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) {
      const int q = __shfl_xor(b, o);
      b = q < b ? q : b;
    }
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      if (i >= per) break;
      if (b == lane + i * 64) v[i] = ninf;
    }
    const float z = expf(m - top);
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

// Fills the lists; the whole workgroup takes part.  out: the workgroup that hands the routing's results out.
template <int THREADS, int BATCH>
__device__ __forceinline__ Lists make_lists(const FewArgs& a, const float* logits, char* smem, bool out) {
  const int pairs = a.T * a.k, entries = a.E_loc + pairs / 16;
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
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int e = tid; e < a.E_loc; e += THREADS) l.mask[e] = 0;
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
    if (id >= 0 && e < (uint32_t)a.E_loc)
      atomicOr(reinterpret_cast<unsigned long long*>(l.mask + e), 1ull << (p / a.k));
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
      int c = own | parts << 16;  // running sums of both (rows <= 2048)
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int q = __shfl_up(c, o);
        if (lane >= o) c += q;
      }
      const int r0 = rows + (c & 0xffff) - own, n0 = n + (c >> 16) - parts;
      if (e < a.E_loc) l.first[e] = r0;
      for (int i = 0; i < parts; ++i) {
        const int left = own - i * BATCH;
        l.entry[n0 + i] = (uint32_t)e | (uint32_t)(left < BATCH ? left : BATCH) << 16;
        l.row[n0 + i] = r0 + i * BATCH;
      }
      const int last = __shfl(c, 63);
      rows += last & 0xffff;
      n += last >> 16;
    }
    if (lane == 0) *total = n;
  }
  __syncthreads();
  // Each row's token and gate weight.  (A choice that names an expert twice has both weights in one row.)
  for (int p = tid; p < pairs; p += THREADS) {
    const int32_t id = l.idx[p];
    const uint32_t e = (uint32_t)id - (uint32_t)a.expert_begin;
    if (id < 0 || e >= (uint32_t)a.E_loc) continue;
    const int t = p / a.k, end = (t + 1) * a.k;
    bool again = false;
    for (int q = t * a.k; q < p; ++q) again |= l.idx[q] == id;
    if (again) continue;
    float w = l.w[p];
    for (int q = p + 1; q < end; ++q) w += l.idx[q] == id ? l.w[q] : 0.f;
    const int r = l.first[e] + __popcll(l.mask[e] & ((1ull << t) - 1));
    l.token[r] = t;
    l.gate[r] = w;
  }
  __syncthreads();
  l.n = *total;
  return l;
}

// A unit of 16 weight rows: 128 reduction indices a row, as a lane holds them.
template <bool FP4>
struct Weights;
template <>
struct Weights<false> {  // step s: indices 32 s + 8 (lane / 16) + 0..7 of row lane % 16
  u32x4 v[4];
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, __amdgpu_buffer_rsrc_t, uint32_t row, int K, int unit, bool in) {
    const int g = (threadIdx.x >> 4) & 3;
    const uint32_t at = row * (uint32_t)(K * 2) + unit * 256 + g * 16;
#pragma unroll
    for (int s = 0; s < 4; ++s) v[s] = __builtin_amdgcn_raw_buffer_load_b128(r, in ? at + s * 64 : kOut, 0, 2);
  }
  __device__ __forceinline__ bf16x8 get(int s) const { return __builtin_bit_cast(bf16x8, v[s]); }
  static __device__ __forceinline__ uint32_t token_at(int unit, int s) { return unit * 256 + s * 64 + ((threadIdx.x >> 4) & 3) * 16; }
};
template <>
struct Weights<true> {  // step s: indices 32 (lane / 16) + 8 s + 0..7 of row lane % 16: a lane has one block
  u32x4 v;
  uint32_t s4;
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, __amdgpu_buffer_rsrc_t rs, uint32_t row, int K, int unit, bool in) {
    const int g = (threadIdx.x >> 4) & 3;
    v = __builtin_amdgcn_raw_buffer_load_b128(r, in ? row * (uint32_t)(K / 2) + unit * 64 + g * 16 : kOut, 0, 2);
    s4 = __builtin_amdgcn_raw_buffer_load_b32(rs, in ? row * (uint32_t)(K / 32) + unit * 4 : kOut, 0, 0);
  }
  __device__ __forceinline__ bf16x8 get(int s) const {
    const float scale = __builtin_bit_cast(float, ((s4 >> (8 * ((threadIdx.x >> 4) & 3))) & 255u) << 23);
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

// ---------------------------------------------------------------------------
// First launch
// ---------------------------------------------------------------------------
// An item is an entry's 16 R rows of the gate (and up) matrix; a workgroup's wavefronts share its reduction and add up
// through LDS.  NB: blocks of 16 tokens of an entry.
template <bool FP4, int NMAT, int NB>
__global__ __launch_bounds__(kUpWaves * 64, NB == 1 ? 4 : 2) void up_kernel(FewArgs a) {
  constexpr int R = FP4 ? 2 : 1, MR = NMAT * R, D = 2;
  constexpr int RED = MR * NB * 256;
  extern __shared__ __attribute__((aligned(16))) char smem[];
  float* red = reinterpret_cast<float*>(smem);
  const Lists l = make_lists<kUpWaves * 64, 16 * NB>(a, a.logits, smem + kUpWaves * RED * 4, blockIdx.x == 0);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  const int blocks = a.F / (16 * R), items = l.n * blocks, units = a.H / kUnit;
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(a.x, (int64_t)a.T * a.H * 2);
  uint16_t* hi = static_cast<uint16_t*>(a.ws);
  uint16_t* lo = hi + (int64_t)a.T * a.k * a.F;
  const void* wp[2] = {a.w0, a.w0_up};
  const uint8_t* sp[2] = {a.s0, a.s0_up};

  for (int item = blockIdx.x; item < items; item += gridDim.x) {
    const int at = item / blocks, f0 = (item - at * blocks) * 16 * R;
    const uint32_t entry = (uint32_t)__builtin_amdgcn_readfirstlane((int)l.entry[at]);
    const int e = entry & 0xffff, n = entry >> 16, first = __builtin_amdgcn_readfirstlane(l.row[at]);
    uint32_t xo[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) xo[b] = b * 16 + l16 < n ? (uint32_t)(l.token[first + b * 16 + l16] * a.H * 2) : kOut;
    const int64_t row0 = (int64_t)e * a.F + f0;
    __amdgpu_buffer_rsrc_t rw[NMAT], rs[NMAT];
#pragma unroll
    for (int m = 0; m < NMAT; ++m) {
      rw[m] = codes_rsrc<FP4>(wp[m], row0, 16 * R, a.H);
      rs[m] = FP4 ? make_rsrc(sp[m] + row0 * (a.H / 32), 16 * R * (a.H / 32)) : rw[m];
    }
    floatx4 acc[MR][NB];
#pragma unroll
    for (int m = 0; m < MR; ++m)
#pragma unroll
      for (int b = 0; b < NB; ++b) acc[m][b] = floatx4{0.f, 0.f, 0.f, 0.f};
    Weights<FP4> w[D][MR];
    u32x4 x[D][NB][4];
    auto load = [&](int q, int u) {
      const bool in = u < units;
#pragma unroll
      for (int m = 0; m < MR; ++m) w[q][m].load(rw[m / R], rs[m / R], (m % R) * 16 + l16, a.H, u, in);
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int s = 0; s < 4; ++s)
          x[q][b][s] = __builtin_amdgcn_raw_buffer_load_b128(rx, in ? xo[b] + Weights<FP4>::token_at(u, s) : kOut, 0, 0);
    };
#pragma unroll
    for (int q = 0; q < D; ++q) load(q, wave + q * kUpWaves);
    for (int u = wave; u < units; u += D * kUpWaves) {
#pragma unroll
      for (int q = 0; q < D; ++q) {
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
          for (int m = 0; m < MR; ++m) {
            const bf16x8 f = w[q][m].get(s);
#pragma unroll
            for (int b = 0; b < NB; ++b)
              acc[m][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f, __builtin_bit_cast(bf16x8, x[q][b][s]), acc[m][b], 0, 0, 0);
          }
        load(q, u + (q + D) * kUpWaves);
      }
    }
    __syncthreads();  // (the last item's sums have been read)
#pragma unroll
    for (int m = 0; m < MR; ++m)
#pragma unroll
      for (int b = 0; b < NB; ++b) *reinterpret_cast<floatx4*>(red + wave * RED + (m * NB + b) * 256 + lane * 4) = acc[m][b];
    __syncthreads();
    // Lane: row l16 of a block of 16 of the entry's, weight rows 4 g + 0..3 of a block of 16.
    for (int q = wave; q < R * NB; q += kUpWaves) {
      const int r = q / NB, b = q % NB, p = b * 16 + l16;
      floatx4 z = {0.f, 0.f, 0.f, 0.f}, u = z;
#pragma unroll
      for (int v = 0; v < kUpWaves; ++v) {
        z += *reinterpret_cast<const floatx4*>(red + v * RED + (r * NB + b) * 256 + lane * 4);
        if (NMAT == 2) u += *reinterpret_cast<const floatx4*>(red + v * RED + ((R + r) * NB + b) * 256 + lane * 4);
      }
      if (p < n) {
        const float gate = l.gate[first + p];
        u32x2 h, m;
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
          uint16_t hh[2], ll[2];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const float y = (NMAT == 2 ? activate(ACT_SILU, z[i + c]) * u[i + c] : activate(ACT_GELU, z[i + c])) * gate;
            hh[c] = f2bf_bits(y);
            const float d = y - bf2f(hh[c]);
            ll[c] = fabsf(d) < __builtin_inff() ? f2bf_bits(d) : 0;  // (an infinity or NaN is all in the first term)
          }
          h[i >> 1] = (uint32_t)hh[0] | (uint32_t)hh[1] << 16;
          m[i >> 1] = (uint32_t)ll[0] | (uint32_t)ll[1] << 16;
        }
        const int64_t o = (int64_t)(first + p) * a.F + f0 + r * 16 + g * 4;
        *reinterpret_cast<u32x2*>(hi + o) = h;
        *reinterpret_cast<u32x2*>(lo + o) = m;
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Second launch
// ---------------------------------------------------------------------------
// A workgroup has 16 R output columns of every token.  Its wavefronts take turns at units of the entries' reductions and
// add each unit's sums to the tokens' in LDS, a copy for each wavefront, so that the order of additions is fixed.
template <bool FP4, int NB, int R>
__global__ __launch_bounds__(kDownWaves * 64, NB == 1 ? 4 : 2) void down_kernel(FewArgs a) {
  constexpr int D = 2, PITCH = 16 * R + 4;
  extern __shared__ __attribute__((aligned(16))) char smem[];
  float* sums = reinterpret_cast<float*>(smem);  // [wavefront][token][PITCH]
  const int each = a.T * PITCH;
  for (int i = threadIdx.x; i < kDownWaves * each / 4; i += kDownWaves * 64)
    reinterpret_cast<floatx4*>(sums)[i] = floatx4{0.f, 0.f, 0.f, 0.f};
  const Lists l = make_lists<kDownWaves * 64, 16 * NB>(a, nullptr, smem + kDownWaves * each * 4, false);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  const int h0 = blockIdx.x * 16 * R, per = a.F / kUnit, units = l.n * per;
  const uint16_t* hi = static_cast<const uint16_t*>(a.ws);
  const int64_t terms = (int64_t)a.T * a.k * a.F;
  float* mine = sums + wave * each;

  struct Unit {
    Weights<FP4> w[R];
    u32x4 hi[NB][4], lo[NB][4];
    int token[NB];  // of this lane's column, -1: none
  };
  Unit q[D];
  auto load = [&](Unit& v, int u) {
    const bool in = u < units;
    const int at = in ? u / per : 0, kf = in ? u - at * per : 0;
    const uint32_t entry = in ? (uint32_t)__builtin_amdgcn_readfirstlane((int)l.entry[at]) : 0;
    const int e = entry & 0xffff, n = entry >> 16, first = in ? __builtin_amdgcn_readfirstlane(l.row[at]) : 0;
    const int64_t row0 = (int64_t)e * a.H + h0;
    const __amdgpu_buffer_rsrc_t rw = codes_rsrc<FP4>(a.w1, row0, 16 * R, a.F);
    const __amdgpu_buffer_rsrc_t rs = FP4 ? make_rsrc(a.s1 + row0 * (a.F / 32), 16 * R * (a.F / 32)) : rw;
#pragma unroll
    for (int r = 0; r < R; ++r) v.w[r].load(rw, rs, r * 16 + l16, a.F, kf, in);
    const __amdgpu_buffer_rsrc_t rh = make_rsrc(hi + (int64_t)first * a.F, (int64_t)n * a.F * 2);
    const __amdgpu_buffer_rsrc_t rl = make_rsrc(hi + terms + (int64_t)first * a.F, (int64_t)n * a.F * 2);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int p = b * 16 + l16;
      v.token[b] = p < n ? l.token[first + p] : -1;
      const uint32_t o = p < n ? (uint32_t)(p * a.F * 2) : kOut;
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        v.hi[b][s] = __builtin_amdgcn_raw_buffer_load_b128(rh, o + Weights<FP4>::token_at(kf, s), 0, 0);
        v.lo[b][s] = __builtin_amdgcn_raw_buffer_load_b128(rl, o + Weights<FP4>::token_at(kf, s), 0, 0);
      }
    }
  };
  auto multiply = [&](const Unit& v) {
    floatx4 acc[R][NB];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int b = 0; b < NB; ++b) acc[r][b] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const bf16x8 f = v.w[r].get(s);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          acc[r][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f, __builtin_bit_cast(bf16x8, v.hi[b][s]), acc[r][b], 0, 0, 0);
          acc[r][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f, __builtin_bit_cast(bf16x8, v.lo[b][s]), acc[r][b], 0, 0, 0);
        }
      }
#pragma unroll
    for (int b = 0; b < NB; ++b)
      if (v.token[b] >= 0)
#pragma unroll
        for (int r = 0; r < R; ++r) *reinterpret_cast<floatx4*>(mine + v.token[b] * PITCH + r * 16 + g * 4) += acc[r][b];
  };
#pragma unroll
  for (int d = 0; d < D; ++d) load(q[d], wave + d * kDownWaves);
  for (int u = wave; u < units; u += D * kDownWaves) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      multiply(q[d]);
      load(q[d], u + (d + D) * kDownWaves);
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < a.T * 4 * R; i += kDownWaves * 64) {
    const int t = i / (4 * R), c = (i - t * 4 * R) * 4;
    floatx4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int v = 0; v < kDownWaves; ++v) o += *reinterpret_cast<const floatx4*>(sums + v * each + t * PITCH + c);
    *reinterpret_cast<floatx4*>(a.out + (int64_t)t * a.H + h0 + c) = o;
  }
}

int cu_count() {
  int dev = 0, n = 0;
  if (hipGetDevice(&dev) != hipSuccess || hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess)
    return 256;
  return n;
}

template <bool FP4, int NB>
hipError_t launch(const FewArgs& a, hipStream_t s) {
  constexpr int R = FP4 ? 2 : 1, R2 = FP4 ? 2 : 1;
  const bool dual = a.w0_up != nullptr;
  const size_t lists = lists_bytes(a.T, a.k, a.E_loc);
  const int64_t items = (int64_t)max_entries(a.T, a.k, a.E_loc, 16 * NB) * (a.F / (16 * R));
  const int64_t most = (int64_t)cu_count() * 4;
  const dim3 grid((unsigned)(items < most ? items : most));
  const size_t red = (size_t)kUpWaves * (dual ? 2 : 1) * R * NB * 1024;
  if (dual) hipLaunchKernelGGL((up_kernel<FP4, 2, NB>), grid, dim3(kUpWaves * 64), red + lists, s, a);
  else hipLaunchKernelGGL((up_kernel<FP4, 1, NB>), grid, dim3(kUpWaves * 64), red + lists, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const size_t sums = (size_t)kDownWaves * a.T * (16 * R2 + 4) * 4;
  hipLaunchKernelGGL((down_kernel<FP4, NB, R2>), dim3((unsigned)(a.H / (16 * R2))), dim3(kDownWaves * 64), sums + lists, s, a);
  return hipGetLastError();
}

}  // namespace

size_t few_tokens_ws_bytes(int T, int k, int F) { return (size_t)T * k * F * 4; }

hipError_t launch_few_tokens(const FewArgs& a, hipStream_t s) {
  const bool wide = a.T > 16 && a.T * a.k > 8 * a.E;
  if (a.s0) return wide ? launch<true, 2>(a, s) : launch<true, 1>(a, s);
  return wide ? launch<false, 2>(a, s) : launch<false, 1>(a, s);
}

}  // namespace moe
