// Dense projection with bias, activation and residual in its epilogue, and its
// gradients.
//
//   forward   z = x . w^T + b;  out = act(z) [* (x . w_up^T + b_up)] + residual
//   backward  dz = d_out * act'(z);  d_x = dz . w;  d_w = dz^T . x;  d_b = sum over the rows of dz
//
// All three products run on one tile scheme, C[m, n] = sum_r A(m, r) * B(n, r)
// with v_mfma_f32_16x16x32_bf16 and fp32 accumulators.  An operand is stored
// either with the reduction index contiguous (rows: x and w in the forward
// product, dz in d_x) or with it outermost (columns: w in d_x, dz and x in
// d_w).  Rows are staged in LDS as 128-byte lines of 64 reduction indices and
// read 16 bytes a lane; columns are staged as stored, 64 reduction indices of
// BM or BN columns, and read with the transposing LDS read (ds_read_b64_tr_b16:
// the 16 lanes of a group, reading 4 rows of 16 columns, each get one column),
// so no operand is transposed in memory.
#include "activation.h"
#include "linear_layout.h"

#include <atomic>
#include <type_traits>

namespace moe {
namespace {

typedef __attribute__((__vector_size__(4 * sizeof(short)))) short s16x4;

// act'(z) (SwiGLU: silu'(z)).
__device__ __forceinline__ float activate_grad(int act, float z) {
  switch (act) {
    case ACT_GELU:
      return 0.5f * (1.0f + erff(z * 0.70710678118654752f)) +
             z * 0.39894228040143268f * __builtin_amdgcn_exp2f(-0.72134752044448170f * z * z);
    case ACT_NONE: return 1.0f;
    default: {
      const float s = sigmoid_f(z);
      return s * (1.0f + z * (1.0f - s));
    }
  }
}

// ---------------------------------------------------------------------------
// Operand staging
// ---------------------------------------------------------------------------
// MFMA fragment (16 operand rows from row c0, 32 reduction indices from 32 ks) of a staged operand: lane holds
// row c0 + lane % 16, reduction indices 32 ks + 8 (lane / 16) + 0..7.
// (paired: the block of 32 rows from c0 on, its fragment `half`).
template <int C>
__device__ __forceinline__ bf16x8 paired_fragment(const char* tile, int c0, int half, int ks, int lane) {
  const int row = c0 + ((lane >> 2) & 3) * 8 + half * 4 + (lane & 3), chunk = ks * 4 + (lane >> 4);
  return *reinterpret_cast<const bf16x8*>(tile + row * 128 + ((chunk ^ swz_p(row)) << 4));
}
template <bool COLS, int C>
__device__ __forceinline__ bf16x8 fragment(const char* tile, int c0, int ks, int lane) {
  const int l16 = lane & 15, g = lane >> 4;
  if constexpr (!COLS) {
    const int row = c0 + l16, chunk = ks * 4 + g;
    return *reinterpret_cast<const bf16x8*>(tile + row * 128 + ((chunk ^ swz(row)) << 4));
  } else {
    const int r = ks * 32 + 8 * g + (l16 >> 2);
    const int chunk = (c0 >> 3) + ((l16 & 3) >> 1);
    const char* p = tile + r * (2 * C) + ((chunk ^ swz_t<C>(r)) << 4) + (l16 & 1) * 8;
    typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
    struct { s16x4 lo, hi; } f;
    f.lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
    const char* p4 = C >= 128 ? p + 8 * C : tile + (r + 4) * (2 * C) + ((chunk ^ swz_t<C>(r + 4)) << 4) + (l16 & 1) * 8;
    f.hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p4);  // row r + 4
    return __builtin_bit_cast(bf16x8, f);
  }
}

struct Operand {
  const uint16_t* p;   // first element
  const uint16_t* p2;  // stages from the second segment on (two weight matrices reduced into one output), or null
  int64_t ld;          // elements between stored rows
  int64_t extent;      // operand rows (m or n); columns operand: stored columns that may be read
  int64_t R;           // reduction length of a segment
};

// Where a tile's results go.
struct Epilogue {
  const float *bias, *bias_up;
  const void* residual;
  void* out;
  uint16_t *z, *z_up;
  int act;
  bool f32;
};

// One output C[m, n] = sum_r A(m, r) * B(n, r), m < M, n < N; b_up: the second matrix of a dual product.
struct Gemm {
  Operand a, b, b_up;
  int64_t M;
  int N;
  int nk, seg;  // stages in all, stages per segment
  int mt, nt;   // tiles
  Epilogue e;
};

// Activation of NV groups of four values (a uniform choice outside the unrolled arithmetic).
template <int NV>
__device__ __forceinline__ void activate_all(int act, floatx4 (&v)[NV], const floatx4 (&u)[NV]) {
  auto each = [&](auto f) {
#pragma unroll
    for (int r = 0; r < NV; ++r)
#pragma unroll
      for (int q = 0; q < 4; ++q) v[r][q] = f(v[r][q], u[r][q]);
  };
  switch (act) {
    case ACT_NONE: break;
    case ACT_GELU: each([](float z, float) { return activate(ACT_GELU, z); }); break;
    case ACT_SILU: each([](float z, float) { return activate(ACT_SILU, z); }); break;
    default: each([](float z, float y) { return activate(ACT_SWIGLU, z) * y; }); break;
  }
}

__device__ __forceinline__ u32x2 pack4(floatx4 x) {
  return u32x2{(uint32_t)f2bf_bits(x[0]) | ((uint32_t)f2bf_bits(x[1]) << 16),
               (uint32_t)f2bf_bits(x[2]) | ((uint32_t)f2bf_bits(x[3]) << 16)};
}

// The rows from row0 on of a product's outputs, and what is added to them: buffer resources that end with row M, so
// that rows past it are neither read nor written (and absent operands read as zeros).  Offsets stay far below 2^31:
// a tile has at most 256 rows of at most 2^20 columns.
struct Sink {
  __amdgpu_buffer_rsrc_t out, z, z_up, res;
  int N, act;
  bool f32, vec, has_z, has_zu, has_res;

  __device__ __forceinline__ Sink(const Epilogue& e, int64_t row0, int rows, int64_t M, int N_) : N(N_), act(e.act), f32(e.f32) {
    const int64_t left = M - row0 < rows ? M - row0 : rows, at = row0 * N, n = left * N;
    vec = (N & 3) == 0;  // then a row's groups of four are aligned
    has_z = e.z != nullptr;
    has_zu = e.z_up != nullptr;
    has_res = e.residual != nullptr;
    const int es = f32 ? 4 : 2;
    out = make_rsrc(static_cast<char*>(e.out) + at * es, n * es);
    res = make_rsrc(static_cast<const char*>(has_res ? e.residual : e.out) + at * es, has_res ? n * es : 0);
    z = make_rsrc((has_z ? e.z : static_cast<uint16_t*>(e.out)) + at, has_z ? n * 2 : 0);
    z_up = make_rsrc((has_zu ? e.z_up : static_cast<uint16_t*>(e.out)) + at, has_zu ? n * 2 : 0);
  }
};

// Four values of one row, cnt of which exist (<= 0: none), at byte offset `at` of row-major data of ES-byte values.
// VEC: rows are whole groups of four, one access each; else value by value.
template <bool VEC, int ES>
__device__ __forceinline__ void put4(__amdgpu_buffer_rsrc_t r, uint32_t at, int cnt, floatx4 x) {
  const u32x2 h = pack4(x);
  if constexpr (VEC) {
    const uint32_t o = cnt > 0 ? at : kOut;
    if constexpr (ES == 2) __builtin_amdgcn_raw_buffer_store_b64(h, r, o, 0, 0);
    else __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, x), r, o, 0, 0);
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t o = q < cnt ? at + q * ES : kOut;
      const float v = x[q];  // (a vector element itself is no object to bit_cast)
      if constexpr (ES == 2) __builtin_amdgcn_raw_buffer_store_b16((uint16_t)(h[q >> 1] >> (16 * (q & 1))), r, o, 0, 0);
      else __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, v), r, o, 0, 0);
    }
  }
}
template <bool VEC, int ES>
__device__ __forceinline__ floatx4 get4(__amdgpu_buffer_rsrc_t r, uint32_t at, int cnt) {
  floatx4 v;
  if constexpr (VEC) {
    const uint32_t o = cnt > 0 ? at : kOut;
    if constexpr (ES == 2) {
      const u32x2 h = __builtin_amdgcn_raw_buffer_load_b64(r, o, 0, 0);
      v = floatx4{bf2f((uint16_t)h[0]), bf2f((uint16_t)(h[0] >> 16)), bf2f((uint16_t)h[1]), bf2f((uint16_t)(h[1] >> 16))};
    } else {
      v = __builtin_bit_cast(floatx4, __builtin_amdgcn_raw_buffer_load_b128(r, o, 0, 0));
    }
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t o = q < cnt ? at + q * ES : kOut;
      v[q] = ES == 2 ? bf2f((uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, o, 0, 0))
                     : __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(r, o, 0, 0));
    }
  }
  return v;
}

// The epilogue of NV rows, r + q * step of the sink, in the four columns from n (a multiple of 4): g and u hold the
// products.  All of the rows' residuals are loaded before the first store.
template <bool VEC, int ES, int NV>
__device__ __forceinline__ void finish(const Sink& k, int r, int step, int n, floatx4 (&g)[NV], floatx4 (&u)[NV],
                                       floatx4 bias, floatx4 bias_up) {
  const int cnt = k.N - n;  // columns that exist
  const uint32_t at = (uint32_t)(r * k.N + n), next = (uint32_t)(step * k.N);  // elements
  floatx4 res[NV];
#pragma unroll
  for (int q = 0; q < NV; ++q) {
    res[q] = floatx4{0.f, 0.f, 0.f, 0.f};
    g[q] += bias;
    u[q] += bias_up;
  }
  if (k.has_res)
#pragma unroll
    for (int q = 0; q < NV; ++q) res[q] = get4<VEC, ES>(k.res, (at + q * next) * ES, cnt);
  if (k.has_z)
#pragma unroll
    for (int q = 0; q < NV; ++q) put4<VEC, 2>(k.z, (at + q * next) * 2, cnt, g[q]);
  if (k.has_zu)
#pragma unroll
    for (int q = 0; q < NV; ++q) put4<VEC, 2>(k.z_up, (at + q * next) * 2, cnt, u[q]);
  activate_all<NV>(k.act, g, u);
#pragma unroll
  for (int q = 0; q < NV; ++q) put4<VEC, ES>(k.out, (at + q * next) * ES, cnt, g[q] + res[q]);
}

// Calls f(VEC, ES) with the sink's access width and output size: one uniform choice ahead of a loop, because code
// that runs once per tile is paid for by its branches and instruction fetches.
template <typename F>
__device__ __forceinline__ void with_layout(const Sink& k, F f) {
  using std::bool_constant;
  using std::integral_constant;
  if (k.vec) {
    if (k.f32) f(bool_constant<true>{}, integral_constant<int, 4>{});
    else f(bool_constant<true>{}, integral_constant<int, 2>{});
  } else {
    if (k.f32) f(bool_constant<false>{}, integral_constant<int, 4>{});
    else f(bool_constant<false>{}, integral_constant<int, 2>{});
  }
}

// Four consecutive biases from column n, zeros past N or where there is none.
__device__ __forceinline__ floatx4 load_bias(const float* b, int n, int N) {
  const __amdgpu_buffer_rsrc_t r = make_rsrc(b, b ? (int64_t)N * 4 : 0);
  floatx4 v;
#pragma unroll
  for (int q = 0; q < 4; ++q)
    v[q] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(r, n + q < N ? (n + q) * 4 : kOut, 0, 0));
  return v;
}

// s_waitcnt lgkmcnt(0), other counters left alone.
__device__ __forceinline__ void wait_lgkm0() { __builtin_amdgcn_s_waitcnt(15 | (7 << 4) | (0 << 8) | (3 << 14)); }

// Workgroup barrier after explicit waits, so that global loads in flight stay in flight across it; the empty asm
// statements keep the compiler from moving memory accesses across.
__device__ __forceinline__ void ring_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// One BM x BN output tile per workgroup (NMAT = 2: BN columns of both matrices), WM x WN wavefronts.
//
// Two LDS buffers and register-staged loads: while stage kt is computed from one buffer, stage kt + 1 goes from
// registers into the other and the registers reload with stage kt + 2.  A stage is four phases, the two halves of
// the wave tile's rows at each of the two 32-wide steps; each phase's fragments are read during the phase before,
// and LDS writes and loads are spread over the MFMAs of the first three.  All of a stage's fragments have been read
// when its last phase begins: there the workgroup synchronises, and the last phase reads the next stage's first
// fragments.  Stages past the end load through a resource of no bytes, so every iteration is the same.
//
// MFMA-bound, under the card's power limit: the SwiGLU product 4096 x 14336 x 4096 (962 GFLOP) takes 0.74-0.8 ms, its
// matrix cores busy 69 % of the cycles at 1.66 GHz; a plain 8192 x 8192 x 8192 product 0.79-0.82 ms, the library's
// 0.76-0.81.  The 16x16x32 MFMA on eight wavefronts keeps every accumulator in VGPRs: four wavefronts with
// 32x32x16 moved them to AGPRs and back (825 us for that SwiGLU product when this took 750-770), eight with 32x32x16
// took 788, and 256x128 tiles on four wavefronts 86 us against 49 at 4096 x 2048 x 2816.
template <int BM, int BN, bool A_COLS, bool B_COLS, int NMAT, int WM, int WN>
struct Tile {
  static constexpr int NW = WM * WN;
  static constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128;
  static constexpr int STAGE = A_BYTES + NMAT * B_BYTES;
  static constexpr int WT_M = BM / WM, WT_N = BN / WN;              // wave tile (per matrix)
  static constexpr int TM = WT_M / 16, TN = WT_N / 16;
  static constexpr int HM = TM / 2, NB = NMAT * TN;                // fragments of half the rows; of the columns
  static constexpr int A_PIECES = BM / (8 * NW), B_PIECES = BN / (8 * NW);  // loads per wavefront and stage
  static constexpr int WP = NMAT * B_PIECES, LOADS = A_PIECES + WP;
  static constexpr int NMFMA = HM * NB;                             // per phase
  static constexpr int PS = (LOADS + 2) / 3;                        // pieces per phase
  static constexpr int PITCH = NMAT * BN + 4;                       // floats per row of the staged result
  static constexpr int SMEM = 2 * STAGE > WM * 32 * PITCH * 4 ? 2 * STAGE : WM * 32 * PITCH * 4;
  static constexpr bool PAIRS = !B_COLS;
  static constexpr int VW = PAIRS ? 2 : 1;                          // groups of four columns side by side in a lane
  static_assert(TN % VW == 0, "pairs of fragments");
  static_assert(HM >= 1 && TN >= 1 && A_PIECES >= 1 && B_PIECES >= 1, "tile too small for the wavefronts");

  // An operand's C rows (columns) from c0 on, as this lane loads them: stage kt through a resource at its first element.
  template <bool COLS, int C, bool PAIRED = false>
  struct Source {
    const char *base, *base2;  // stage 0 of the two segments (base2 less the first segment's stages)
    SourceMap<COLS, C, NW, PAIRED> map;
    uint32_t off, step;

    __device__ __forceinline__ Source(const Operand& o, int64_t c0, int seg, int k1, int wave, int lane)
        : map(o.ld, o.extent, o.R, c0, seg, k1, wave, lane), off(map.off), step(map.step) {
      base = reinterpret_cast<const char*>(o.p + (COLS ? c0 : c0 * o.ld));
      base2 = o.p2 ? reinterpret_cast<const char*>(o.p2 + (COLS ? c0 : c0 * o.ld)) - seg * map.adv : nullptr;
    }
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(int kt) const {
      const bool second = base2 && kt >= map.seg;
      return make_rsrc((second ? base2 : base) + kt * map.adv, map.bytes(kt));
    }
    __device__ __forceinline__ uint32_t offset(int kt) const { return map.offset(kt); }
  };

  struct Stage {  // where a stage's loads come from
    __amdgpu_buffer_rsrc_t a, b, bu;
    uint32_t oa, ob;
  };

  // VW groups of four values side by side, at byte offset `at` (kOut and above: none).
  template <int ES>
  static __device__ __forceinline__ void put(__amdgpu_buffer_rsrc_t r, uint32_t at, const floatx4 (&v)[VW]) {
    if constexpr (ES == 2 && VW == 2) {
      const u32x2 a = pack4(v[0]), b = pack4(v[1]);
      __builtin_amdgcn_raw_buffer_store_b128(u32x4{a[0], a[1], b[0], b[1]}, r, at, 0, 0);
    } else {
#pragma unroll
      for (int q = 0; q < VW; ++q) put4<true, ES>(r, at + q * 4 * ES, 1, v[q]);
    }
  }
  template <int ES>
  static __device__ __forceinline__ void get(__amdgpu_buffer_rsrc_t r, uint32_t at, floatx4 (&v)[VW]) {
    if constexpr (ES == 2 && VW == 2) {
      const u32x4 h = __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, 0);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        v[q >> 1][(q & 1) * 2] = bf2f((uint16_t)h[q]);
        v[q >> 1][(q & 1) * 2 + 1] = bf2f((uint16_t)(h[q] >> 16));
      }
    } else {
#pragma unroll
      for (int q = 0; q < VW; ++q) v[q] = get4<true, ES>(r, at + q * 4 * ES, 1);
    }
  }

  // The epilogue straight from the accumulators: a lane holds, for row r + 16 i, the 4 VW columns from n + 16 VW j on.
  // For products without an activation and SwiGLU, where rows are whole pieces: 12.5 us against the LDS epilogue's 17
  // at 4096 x 4096 x 64 (22 there with GELU, 19 with SiLU), 62 against 84 at 4096 x 14336 x 64 (SwiGLU), 93 against 104
  // there with z and z_up saved (with single groups of four bf16 values 126, which is why the forward product pairs its
  // fragments).
  template <int ES>
  static __device__ __forceinline__ void direct(const Sink& k, const Gemm& g, int r, int n, floatx4 (&acc)[NB][TM]) {
    asm volatile("" : "+v"(r), "+v"(n));                       // nothing of this ahead of the branch to it
    constexpr int P = TN / VW;                                 // pieces of a row
    constexpr int AHEAD = TM * NB <= 16 ? 1 : 0;               // residual rows are loaded ahead while registers last,
    constexpr int TOGETHER = (AHEAD ? 8 : 4) / TN;             // this many together
    constexpr int C = TM < TOGETHER ? TM : TOGETHER, CH = TM / C;
    uint32_t at[P];
    floatx4 b[NB];
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int col = n + 16 * VW * p;
      at[p] = col < k.N ? (uint32_t)((r * k.N + col) * ES) : kOut;
#pragma unroll
      for (int q = 0; q < VW; ++q) {
        b[p * VW + q] = load_bias(g.e.bias, col + 4 * q, k.N);
        if (NMAT == 2) b[NB - TN + p * VW + q] = load_bias(g.e.bias_up, col + 4 * q, k.N);
      }
    }
    const uint32_t step = (uint32_t)(16 * k.N * ES);
    floatx4 res[AHEAD + 1][C][P][VW];
    auto load = [&](int c, uint32_t from) {  // chunk c, `from` bytes past at[]
#pragma unroll
      for (int i = 0; i < C; ++i)
#pragma unroll
        for (int p = 0; p < P; ++p) get<ES>(k.res, at[p] + from + i * step, res[c & AHEAD][i][p]);
    };
    auto all = [&](auto has_res, auto has_z) {
#pragma unroll
      for (int j = 0; j < NB; ++j) asm volatile("" : "+v"(b[j]));
      if constexpr (has_res && AHEAD) load(0, 0);
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        if constexpr (has_res)
          if (c + AHEAD < CH) load(c + AHEAD, AHEAD * C * step);
#pragma unroll
        for (int i = 0; i < C; ++i)
#pragma unroll
          for (int p = 0; p < P; ++p) {
            const uint32_t here = at[p] + i * step, z_at = here / (ES / 2);  // (past every resource where at[] is)
            floatx4 v[VW], u[VW];
#pragma unroll
            for (int q = 0; q < VW; ++q) {
              v[q] = acc[p * VW + q][c * C + i] + b[p * VW + q];
              u[q] = NMAT == 2 ? acc[NB - TN + p * VW + q][c * C + i] + b[NB - TN + p * VW + q] : v[q];
            }
            if constexpr (has_z) {
              put<2>(k.z, z_at, v);
              if (NMAT == 2) put<2>(k.z_up, z_at, u);
            }
#pragma unroll
            for (int q = 0; q < VW; ++q) {
              if constexpr (NMAT == 2)
#pragma unroll
                for (int e = 0; e < 4; ++e) v[q][e] = activate(ACT_SWIGLU, v[q][e]) * u[q][e];
              if constexpr (has_res) v[q] += res[c & AHEAD][i][p][q];
            }
            put<ES>(k.out, here, v);
          }
#pragma unroll
        for (int p = 0; p < P; ++p) {
          at[p] += C * step;
          asm volatile("" : "+v"(at[p]));  // (all chunks' addresses at once would not fit)
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    using std::false_type;
    using std::true_type;
    if (k.has_z || k.has_zu) {  // (stores of the one that is absent go nowhere)
      if (k.has_res) all(true_type{}, true_type{});
      else all(false_type{}, true_type{});
    } else {
      if (k.has_res) all(true_type{}, false_type{});
      else all(false_type{}, false_type{});
    }
  }

  static __device__ __forceinline__ void run(char* smem, const Gemm& g, int64_t m0, int n0, int k0, int k1,
                                             float* part) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const Source<A_COLS, BM> src_a(g.a, m0, A_COLS ? g.seg : g.nk, k1, wave, lane);
    const Source<B_COLS, BN, PAIRS> src_b(g.b, n0, g.seg, k1, wave, lane);
    const Source<B_COLS, BN, PAIRS> src_u(NMAT == 2 ? g.b_up : g.b, n0, g.seg, k1, wave, lane);
    floatx4 acc[NB][TM];
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int i = 0; i < TM; ++i) acc[j][i] = floatx4{0.f, 0.f, 0.f, 0.f};

    u32x4 stg[LOADS];
    auto stage_a = [&](Stage& st, int kt) {
      st.a = src_a.rsrc(kt);
      st.oa = src_a.offset(kt);
    };
    auto stage_b = [&](Stage& st, int kt) {
      st.b = src_b.rsrc(kt);
      if (NMAT == 2) st.bu = src_u.rsrc(kt);
      st.ob = src_b.offset(kt);
    };
    auto vload = [&](int p, const Stage& st) {
      if (p < A_PIECES) {
        stg[p] = __builtin_amdgcn_raw_buffer_load_b128(st.a, st.oa + p * src_a.step, 0, 0);
      } else {
        const int pb = p - A_PIECES, m = pb / B_PIECES, q = pb % B_PIECES;
        stg[p] = __builtin_amdgcn_raw_buffer_load_b128(m ? st.bu : st.b, st.ob + q * src_b.step, 0, 0);
      }
    };
    auto vwrite = [&](int p, int buf) {
      const int pb = p - A_PIECES;
      const int line = p < A_PIECES ? p * NW : (A_BYTES + (pb / B_PIECES) * B_BYTES) / 1024 + (pb % B_PIECES) * NW;
      *reinterpret_cast<u32x4*>(smem + buf * STAGE + (line + wave) * 1024 + lane * 16) = stg[p];
    };
    bf16x8 fa[2][HM], fb[2][NB];  // rows: by half of the wave tile; columns: by step
    auto read_a = [&](int half, int buf, int ks) {
#pragma unroll
      for (int i = 0; i < HM; ++i)
        fa[half][i] = fragment<A_COLS, BM>(smem + buf * STAGE, wm * WT_M + (half * HM + i) * 16, ks, lane);
    };
    auto read_b = [&](int buf, int ks) {
#pragma unroll
      for (int j = 0; j < NB; ++j)
        if constexpr (PAIRS)
          fb[ks][j] = paired_fragment<BN>(smem + buf * STAGE + A_BYTES + (j / TN) * B_BYTES, wn * WT_N + (j % TN) / 2 * 32, j & 1, ks, lane);
        else
          fb[ks][j] = fragment<B_COLS, BN>(smem + buf * STAGE + A_BYTES + (j / TN) * B_BYTES, wn * WT_N + (j % TN) * 16, ks, lane);
    };
    // The MFMAs of one phase.  They have no side effects: the use of the accumulators keeps them ahead of the next
    // phase's.
    auto mfmas = [&](int half, int ks) {
#pragma unroll
      for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int i = 0; i < HM; ++i)
          acc[j][half * HM + i] =
              __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[ks][j], fa[half][i], acc[j][half * HM + i], 0, 0, 0);
#pragma unroll
      for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int i = 0; i < HM; ++i) asm volatile("" : "+v"(acc[j][half * HM + i]));
    };
    // Instruction order of a phase with nr LDS reads and np pieces (a write and a load each): one of them after
    // each MFMA.
    auto order = [&](auto nr_, auto np_) {
      constexpr int nr = decltype(nr_)::value, np = decltype(np_)::value;
#pragma unroll
      for (int t = 0; t < NMFMA || t < nr + 2 * np; ++t) {
        if (t < NMFMA) __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        if (t < nr) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        else if (t < nr + 2 * np) {
          if ((t - nr) % 2 == 0) __builtin_amdgcn_sched_group_barrier(0x200, 1, 0);
          else __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    constexpr int RA = HM * (A_COLS ? 2 : 1), RB = NB * (B_COLS ? 2 : 1);
    constexpr int P0 = PS < LOADS ? PS : LOADS, P1 = 2 * PS < LOADS ? 2 * PS : LOADS;
    using std::integral_constant;

    // Prologue: stage k0 into buffer 0, stage k0 + 1 into the registers.
    Stage st;
    stage_a(st, k0);
    stage_b(st, k0);
#pragma unroll
    for (int p = 0; p < LOADS; ++p) vload(p, st);
#pragma unroll
    for (int p = 0; p < LOADS; ++p) vwrite(p, 0);
    stage_a(st, k0 + 1);
    stage_b(st, k0 + 1);
#pragma unroll
    for (int p = 0; p < LOADS; ++p) vload(p, st);
    wait_lgkm0();
    ring_barrier();
    read_a(0, 0, 0);
    read_b(0, 0);

    for (int kt = k0; kt < k1; ++kt) {
      const int buf = (kt - k0) & 1, wbuf = buf ^ 1;
      stage_a(st, kt + 2);
      stage_b(st, kt + 2);
      auto pieces = [&](int from, int to) {
#pragma unroll
        for (int p = 0; p < LOADS; ++p)
          if (p >= from && p < to) {
            vwrite(p, wbuf);
            vload(p, st);
          }
      };
      read_a(1, buf, 0);
      pieces(0, P0);
      mfmas(0, 0);
      order(integral_constant<int, RA>{}, integral_constant<int, P0>{});
      read_a(0, buf, 1);
      read_b(buf, 1);
      pieces(P0, P1);
      mfmas(1, 0);
      order(integral_constant<int, RA + RB>{}, integral_constant<int, P1 - P0>{});
      read_a(1, buf, 1);
      pieces(P1, LOADS);
      mfmas(0, 1);
      order(integral_constant<int, RA>{}, integral_constant<int, LOADS - P1>{});
      wait_lgkm0();    // this wavefront's reads of stage kt and writes of stage kt + 1 are complete
      ring_barrier();  // stage kt + 1 is visible to all; the buffer of stage kt is free
      __builtin_amdgcn_sched_barrier(0);
      read_a(0, wbuf, 0);
      read_b(wbuf, 0);
      mfmas(1, 1);
      order(integral_constant<int, RA + RB>{}, integral_constant<int, 0>{});
    }

    const Sink sink(g.e, m0, BM, g.M, g.N);
    if (!part && (g.N & (4 * VW - 1)) == 0 && (NMAT == 2 || sink.act == ACT_NONE)) {
      const int r = wm * WT_M + (lane & 15), n = n0 + wn * WT_N + (lane >> 4) * 4 * VW;
      if (sink.f32) direct<4>(sink, g, r, n, acc);
      else direct<2>(sink, g, r, n, acc);
      return;
    }

    // The other epilogues (GELU and SiLU, whose code would be long unrolled; split sums; rows of odd lengths, whose
    // values go one by one): 32 rows of each wavefront row at a time through LDS, so that global memory is accessed
    // along rows.  The columns' side feeds the MFMA's rows, so a lane holds, for row lane % 16 of a 16-row block,
    // columns 4 (lane / 16) + 0..3 of a 16-column block (paired: 8 (lane / 16) + 0..3 or 4..7 of 32 columns).
    float* sm = reinterpret_cast<float*>(smem);
    constexpr int C4 = BN / 4, STEP = NW * 64 / C4, NV = 32 / STEP < 4 ? 32 / STEP : 4;  // a thread keeps its columns
    const int n = (threadIdx.x % C4) * 4;
    const floatx4 bias = load_bias(g.e.bias, n0 + n, g.N), bias_up = load_bias(g.e.bias_up, n0 + n, g.N);
#pragma unroll 1
    for (int i = 0; i < TM / 2; ++i) {
      // (barriers that wait for LDS alone: __syncthreads() would also wait for the last pass's stores, 1.5 us)
      wait_lgkm0();
      ring_barrier();
#pragma unroll
      for (int ii = 0; ii < TM / 2; ++ii) {
        if (ii != i) continue;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < NB; ++j) {
            const int c = (j / TN) * BN + wn * WT_N + (j % TN) / VW * 16 * VW + (lane >> 4) * 4 * VW + j % VW * 4;
            *reinterpret_cast<floatx4*>(sm + (wm * 32 + h * 16 + (lane & 15)) * PITCH + c) = acc[j][2 * ii + h];
          }
      }
      wait_lgkm0();
      ring_barrier();
      // NV rows of this thread's columns at a time.
      auto rows = [&](auto f) {
#pragma unroll 1
        for (int h = 0; h < WM; ++h)
#pragma unroll 1
          for (int r0 = 0; r0 < 32; r0 += NV * STEP) {
            floatx4 v[NV], u[NV];
            const int rt = r0 + threadIdx.x / C4;
#pragma unroll
            for (int r = 0; r < NV; ++r) {
              const float* p = sm + (h * 32 + rt + r * STEP) * PITCH + n;
              v[r] = *reinterpret_cast<const floatx4*>(p);
              u[r] = NMAT == 2 ? *reinterpret_cast<const floatx4*>(p + BN) : floatx4{0.f, 0.f, 0.f, 0.f};
            }
            f(h * WT_M + i * 32 + rt, v, u);
          }
      };
      if (part) {
        rows([&](int r, floatx4 (&v)[NV], floatx4 (&u)[NV]) {
#pragma unroll
          for (int q = 0; q < NV; ++q) {
            float* o = part + (int64_t)(r + q * STEP) * (NMAT * BN) + n;
            *reinterpret_cast<floatx4*>(o) = v[q];
            if (NMAT == 2) *reinterpret_cast<floatx4*>(o + BN) = u[q];
          }
        });
      } else {
        with_layout(sink, [&](auto vec, auto es) {
          rows([&](int r, floatx4 (&v)[NV], floatx4 (&u)[NV]) {
            finish<decltype(vec)::value, decltype(es)::value, NV>(sink, r, STEP, n0 + n, v, u, bias, bias_up);
          });
        });
      }
    }
  }
};

constexpr int kXcds = 8;
constexpr int kGroupM = 8;  // row tiles per rasterisation group

// Workgroup -> slice and tile: workgroups go round-robin to the XCDs, and each XCD's run is contiguous in an order of
// slices, and in a slice of groups of kGroupM row tiles, column by column, so that tiles that run together share
// operand panels in its L2.
__device__ __forceinline__ void tile_of(int bid, int G, int mt, int nt, int tiles, int& slice, int& ti, int& tj) {
  const int each = G / kXcds, more = G % kXcds, x = bid % kXcds;
  int vid = x * each + (x < more ? x : more) + bid / kXcds;
  slice = vid / tiles;
  vid -= slice * tiles;
  const int per = kGroupM * nt, grp = vid / per, rem = vid % per;
  const int rows = mt - grp * kGroupM < kGroupM ? mt - grp * kGroupM : kGroupM;
  tj = rem / rows;
  ti = grp * kGroupM + rem % rows;
}

template <int KIND, bool A_COLS, bool B_COLS, int NMAT>
using KindTile = Tile<kKinds[KIND].bm, kKinds[KIND].bn / NMAT, A_COLS, B_COLS, NMAT, kKinds[KIND].wm, kKinds[KIND].wn>;

// One product of a launch: its tiles times S slices of the reduction, slice q covering stages
// [q nk / S, (q + 1) nk / S).  With S > 1 slice q of tile t leaves fp32 sums at part + (q tiles + t) (tile floats),
// which reduce_kernel adds in order.
struct Job {
  Gemm g;
  int S;
  int first;  // first workgroup
  float* part;
};

template <int KIND, bool A_COLS, bool B_COLS, int NMAT>
__device__ __forceinline__ void run_job(char* smem, const Job& j, int bid) {
  using T = KindTile<KIND, A_COLS, B_COLS, NMAT>;
  constexpr int BM = kKinds[KIND].bm, BN = kKinds[KIND].bn / NMAT;
  const int tiles = j.g.mt * j.g.nt;
  int ti, tj, q;
  tile_of(bid, tiles * j.S, j.g.mt, j.g.nt, tiles, q, ti, tj);
  const int k0 = (int)((int64_t)q * j.g.nk / j.S), k1 = (int)((int64_t)(q + 1) * j.g.nk / j.S);
  float* part = j.S > 1 ? j.part + ((int64_t)q * tiles + ti * j.g.nt + tj) * (BM * NMAT * BN) : nullptr;
  T::run(smem, j.g, (int64_t)ti * BM, tj * BN, k0, k1, part);
}

template <int KIND, int NMAT>
__global__ __launch_bounds__(kKinds[KIND].threads(), KIND == 3 ? 3 : 2) void forward_kernel(Job j) {
  __shared__ __attribute__((aligned(1024))) char smem[KindTile<KIND, false, false, NMAT>::SMEM];
  run_job<KIND, false, false, NMAT>(smem, j, blockIdx.x);
}

// ---------------------------------------------------------------------------
// Few rows: stream the weights
// ---------------------------------------------------------------------------
// M <= 16.  A workgroup owns 16 weight rows -- 16 output columns, or 8 of the gate's and the same 8 of the up
// matrix's -- and its NK wavefronts a share of K each, so nothing is exchanged before the end.  A load takes 128
// bytes of each of 8 rows: with 64 bytes of 16 rows, the MFMA's own layout, whole lines are asked for twice and a CU
// draws 20 GB/s instead of 28 (1 x 28672 x 8192: 92 against 67 us).  So a wavefront passes its operands through LDS
// of its own, which needs no barrier (its LDS accesses complete in order).  U steps of 64 reduction indices are in
// flight.  Bound by the weights' bytes: 58.7 MB at 1 x 2048 x 7168 (SwiGLU) in 10.1 us, 5.8 TB/s.  The wavefronts'
// sums meet in LDS and are added in order.
template <bool DUAL, int NK, int U>
__global__ __launch_bounds__(NK * 64) void skinny_kernel(Gemm g) {
  constexpr int COLS = DUAL ? 8 : 16;  // output columns
  __shared__ __attribute__((aligned(1024))) char smem[NK * 4096];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  char* sw = smem + wave * 4096;  // weight rows, then token rows: 16 x 128 B each, chunks swizzled
  char* sx = sw + 2048;
  const int n0 = blockIdx.x * COLS;
  const int K = (int)g.b.R, steps = (K + BK - 1) / BK, M = (int)g.M;
  const int s0 = (int)((int64_t)wave * steps / NK), s1 = (int)((int64_t)(wave + 1) * steps / NK);
  const int cols = g.N - n0 < COLS ? g.N - n0 : COLS;
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(g.a.p, (int64_t)M * K * 2);
  const __amdgpu_buffer_rsrc_t rw = make_rsrc(g.b.p + (int64_t)n0 * K, (int64_t)cols * K * 2);
  const __amdgpu_buffer_rsrc_t ru = DUAL ? make_rsrc(g.b_up.p + (int64_t)n0 * K, (int64_t)cols * K * 2) : rw;
  const int r = lane >> 3;
  const int k0 = ((lane & 7) ^ swz(r)) * 8, k1 = ((lane & 7) ^ swz(r + 8)) * 8;  // this lane's chunk of rows r, r + 8
  const uint32_t w0 = r < cols ? (r * K + k0) * 2 : kOut;
  const uint32_t w1 = DUAL ? (r < cols ? (r * K + k1) * 2 : kOut) : (r + 8 < cols ? ((r + 8) * K + k1) * 2 : kOut);
  const uint32_t x0 = r < M ? (r * K + k0) * 2 : kOut, x1 = r + 8 < M ? ((r + 8) * K + k1) * 2 : kOut;
  struct Step {
    u32x4 w0, w1, x0, x1;
  };
  auto load = [&](Step& b, int s) {
    const int kk = s * BK;
    const bool in0 = s < s1 && kk + k0 < K, in1 = s < s1 && kk + k1 < K;
    b.w0 = __builtin_amdgcn_raw_buffer_load_b128(rw, in0 && w0 != kOut ? w0 + kk * 2 : kOut, 0, 2);
    b.w1 = __builtin_amdgcn_raw_buffer_load_b128(ru, in1 && w1 != kOut ? w1 + kk * 2 : kOut, 0, 2);
    b.x0 = __builtin_amdgcn_raw_buffer_load_b128(rx, in0 && x0 != kOut ? x0 + kk * 2 : kOut, 0, 0);
    if (M > 8) b.x1 = __builtin_amdgcn_raw_buffer_load_b128(rx, in1 && x1 != kOut ? x1 + kk * 2 : kOut, 0, 0);
  };
  if (M <= 8) *reinterpret_cast<u32x4*>(sx + 1024 + lane * 16) = u32x4{0, 0, 0, 0};
  floatx4 acc = {0.f, 0.f, 0.f, 0.f};
  auto multiply = [&](const Step& b) {
    *reinterpret_cast<u32x4*>(sw + lane * 16) = b.w0;
    *reinterpret_cast<u32x4*>(sw + 1024 + lane * 16) = b.w1;
    *reinterpret_cast<u32x4*>(sx + lane * 16) = b.x0;
    if (M > 8) *reinterpret_cast<u32x4*>(sx + 1024 + lane * 16) = b.x1;
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fragment<false, 16>(sw, 0, ks, lane), fragment<false, 16>(sx, 0, ks, lane),
                                                    acc, 0, 0, 0);
  };
  Step b[U];
#pragma unroll
  for (int q = 0; q < U; ++q) load(b[q], s0 + q);
  for (int s = s0; s < s1; s += U)
#pragma unroll
    for (int q = 0; q < U; ++q) {
      multiply(b[q]);
      load(b[q], s + q + U);
    }
  __syncthreads();
  floatx4* part = reinterpret_cast<floatx4*>(smem);
  part[wave * 64 + lane] = acc;
  __syncthreads();
  // Lane l of a partial sum: token row l % 16, weight rows 4 (l / 16) + 0..3.
  if (threadIdx.x < (DUAL ? 32 : 64)) {
    floatx4 v[1] = {part[lane]}, u[1] = {part[DUAL ? lane + 32 : lane]};
    for (int q = 1; q < NK; ++q) {
      v[0] += part[q * 64 + lane];
      u[0] += part[q * 64 + (DUAL ? lane + 32 : lane)];
    }
    const int n = n0 + (lane >> 4) * 4;
    const Sink sink(g.e, 0, 16, g.M, g.N);
    with_layout(sink, [&](auto vec, auto es) {
      finish<decltype(vec)::value, decltype(es)::value, 1>(sink, lane & 15, 0, n, v, u, load_bias(g.e.bias, n, g.N),
                                                           load_bias(g.e.bias_up, n, g.N));
    });
  }
}

// ---------------------------------------------------------------------------
// dz, and the bias gradients
// ---------------------------------------------------------------------------
constexpr int kDzRows = 8;  // rows per block of dz_kernel

// VEC consecutive values of row-major [., N] data as floats (VEC = 8: 16-byte aligned).
template <int VEC>
__device__ __forceinline__ void load_values(float (&v)[VEC], const void* p, bool f32, int64_t at) {
  if constexpr (VEC == 1) {
    v[0] = f32 ? static_cast<const float*>(p)[at] : bf2f(static_cast<const uint16_t*>(p)[at]);
  } else if (f32) {
    const floatx4* q = reinterpret_cast<const floatx4*>(static_cast<const float*>(p) + at);
    const floatx4 a = __builtin_nontemporal_load(q), b = __builtin_nontemporal_load(q + 1);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] = a[e];
      v[4 + e] = b[e];
    }
  } else {
    const u32x4 a = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p) + at));
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[2 * e] = bf2f((uint16_t)a[e]);
      v[2 * e + 1] = bf2f((uint16_t)(a[e] >> 16));
    }
  }
}

template <int VEC>
__device__ __forceinline__ void store_values(uint16_t* o, const float (&v)[VEC]) {
  if constexpr (VEC == 1) {
    *o = f2bf_bits(v[0]);
  } else {
    u32x4 h;
#pragma unroll
    for (int e = 0; e < 4; ++e) h[e] = (uint32_t)f2bf_bits(v[2 * e]) | ((uint32_t)f2bf_bits(v[2 * e + 1]) << 16);
    *reinterpret_cast<u32x4*>(o) = h;
  }
}

// dz (SwiGLU: dz and dz_up, dz_up at column offset Np) rounded to bf16, [M, ld] with zeros in columns [N, Np) of
// each, and the block's column sums of the unrounded values, part[block row][mats][N].  bf16 because the matrix
// instructions take it, like the products' other operands: the gradients' relative error against 64 bits is then
// 2.3e-3, of which their own rounding is 1.7e-3 (two independent roundings of that size: sqrt 2 of it); dz in two bf16
// parts would leave 1.7e-3 and double the products.  HBM-bound: reads d_out, z
// (and z_up), writes dz once.  64 threads side by side of VEC columns (8 where rows are 16-byte aligned, N % 8 ==
// 0), four rows apart; each thread has the loads of its two rows in flight and ends.  Blocks of 32 rows, two at a
// time, took 10 us against 4 at 197 x 1000 and 43 against 33 at 8192 x 2816 (SwiGLU).
template <int VEC>
__global__ __launch_bounds__(256) void dz_kernel(const void* __restrict__ d_out, bool f32,
                                                 const uint16_t* __restrict__ z, const uint16_t* __restrict__ z_up,
                                                 int act, int64_t M, int N, int Np, int ld, uint16_t* __restrict__ dz,
                                                 float* __restrict__ part) {
  constexpr int U = kDzRows / 4;
  const int n = (blockIdx.x * 64 + (threadIdx.x & 63)) * VEC, rg = threadIdx.x >> 6;
  const int64_t r0 = (int64_t)blockIdx.y * kDzRows + rg;
  const bool dual = act == ACT_SWIGLU, in = n < N;
  float g[U][VEC], a[U][VEC], b[U][VEC];
#pragma unroll
  for (int q = 0; q < U; ++q) {
    const int64_t r = r0 + q * 4;
#pragma unroll
    for (int e = 0; e < VEC; ++e) g[q][e] = a[q][e] = b[q][e] = 0.f;
    if (in && r < M) {
      load_values<VEC>(g[q], d_out, f32, r * N + n);
      if (act != ACT_NONE) load_values<VEC>(a[q], z, false, r * N + n);
      if (dual) load_values<VEC>(b[q], z_up, false, r * N + n);
    }
  }
  auto each = [&](auto f) {
#pragma unroll
    for (int q = 0; q < U; ++q)
#pragma unroll
      for (int e = 0; e < VEC; ++e) f(g[q][e], a[q][e], b[q][e]);
  };
  // g becomes dz and b becomes dz_up.
  switch (act) {
    case ACT_NONE: break;
    case ACT_GELU: each([](float& d, float& zz, float&) { d *= activate_grad(ACT_GELU, zz); }); break;
    case ACT_SILU: each([](float& d, float& zz, float&) { d *= activate_grad(ACT_SILU, zz); }); break;
    default:
      each([](float& d, float& zz, float& u) {
        const float go = d;
        d = go * activate_grad(ACT_SWIGLU, zz) * u;
        u = go * activate(ACT_SWIGLU, zz);
      });
  }
  float s0[VEC], s1[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) s0[e] = s1[e] = 0.f;
#pragma unroll
  for (int q = 0; q < U; ++q) {
    const int64_t r = r0 + q * 4;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      s0[e] += g[q][e];
      s1[e] += b[q][e];
    }
    if (n < Np && r < M) {
      store_values<VEC>(dz + r * ld + n, g[q]);
      if (dual) store_values<VEC>(dz + r * ld + Np + n, b[q]);
    }
  }
  if (!part) return;
  __shared__ float sums[4][2][64 * VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    sums[rg][0][(threadIdx.x & 63) * VEC + e] = s0[e];
    sums[rg][1][(threadIdx.x & 63) * VEC + e] = s1[e];
  }
  __syncthreads();
  const int mats = dual ? 2 : 1;
  for (int c = threadIdx.x; c < mats * 64 * VEC; c += 256) {
    const int m = c / (64 * VEC), x = c % (64 * VEC), col = blockIdx.x * 64 * VEC + x;
    if (col < N)
      part[((int64_t)blockIdx.y * mats + m) * N + col] =
          (sums[0][m][x] + sums[1][m][x]) + (sums[2][m][x] + sums[3][m][x]);
  }
}

// Column sums of dz_kernel's blocks: 64 columns a workgroup, an equal share of the row blocks for each of its
// wavefronts, 16 of them in flight, added in order.
struct BiasSums {
  const float* part;
  int64_t rows;  // row blocks
  int N, mats;
  float *d_bias, *d_bias_up;
};
__device__ __forceinline__ void bias_sum(char* smem, const BiasSums& b, int bid) {
  float* sm = reinterpret_cast<float*>(smem);
  const int c = bid * 64 + (threadIdx.x & 63), q = threadIdx.x >> 6, waves = blockDim.x >> 6, width = b.mats * b.N;
  float s[4] = {0.f, 0.f, 0.f, 0.f};
  if (c < width) {
    int64_t r = q * b.rows / waves;
    const int64_t end = (q + 1) * b.rows / waves;
    const float* p = b.part + c;
    for (; r + 16 <= end; r += 16) {
      float v[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) v[e] = p[(r + e) * width];
#pragma unroll
      for (int e = 0; e < 16; ++e) s[e & 3] += v[e];
    }
    for (; r < end; ++r) s[0] += p[r * width];
  }
  sm[threadIdx.x] = (s[0] + s[1]) + (s[2] + s[3]);
  __syncthreads();
  if (q == 0 && c < width) {
    float v = sm[threadIdx.x];
    for (int w = 1; w < waves; ++w) v += sm[64 * w + threadIdx.x];
    float* o = c < b.N ? b.d_bias : b.d_bias_up;
    if (o) o[c < b.N ? c : c - b.N] = v;
  }
}

// The backward pass's products in one launch (8192 x 2816 x 2048 SwiGLU, 378 GFLOP: 330-350 us, MFMA 55 % busy at 2.0
// GHz, because 432 tiles of 88 and 128 stages leave 80 CUs without a second one; splitting the weight gradients to
// even that out would write and read 100-180 MB of partial tiles), so that the tiles of one fill the CUs that another
// leaves idle: the input gradient (rows, columns; jobs 0 .. nx - 1, at most one; ahead of the others by 2-4 % at 8192 x 2816 x 2048),
// the weight gradients (both operands columns) and the bias gradients (from workgroup bias_first on).
struct BackwardJobs {
  Job j[3];
  int n, nx, bias_first;
  BiasSums bias;
};

template <int KIND>
__global__ __launch_bounds__(kKinds[KIND].threads(), KIND == 3 ? 3 : 2) void backward_kernel(BackwardJobs b) {
  using TW = KindTile<KIND, true, true, 1>;
  using TX = KindTile<KIND, false, true, 1>;
  __shared__ __attribute__((aligned(1024))) char smem[TW::SMEM > TX::SMEM ? TW::SMEM : TX::SMEM];
  if ((int)blockIdx.x >= b.bias_first) {
    bias_sum(smem, b.bias, blockIdx.x - b.bias_first);
    return;
  }
  int q = 0;
  while (q + 1 < b.n && (int)blockIdx.x >= b.j[q + 1].first) ++q;
  const int bid = blockIdx.x - b.j[q].first;
  if (q >= b.nx) run_job<KIND, true, true, 1>(smem, b.j[q], bid);
  else run_job<KIND, false, true, 1>(smem, b.j[q], bid);
}

// Adds the slices of a job's tiles in order and applies its epilogue; one group of four outputs per thread.  The
// partial tiles come from the last-level cache (64 x 4096 x 1024, backward: 5 us, with launch).
__device__ __forceinline__ void reduce_job(const Job& j, int bm, int bn, int nmat) {
  const int n4 = (j.g.N + 3) / 4;
  const int64_t o = blockIdx.x * 256ll + threadIdx.x;
  if (j.S <= 1 || o >= j.g.M * n4) return;
  const int64_t row = o / n4;
  const int n = (int)(o - row * n4) * 4;
  const int64_t tiles = (int64_t)j.g.mt * j.g.nt, size = (int64_t)bm * nmat * bn;
  const float* p = j.part + (row / bm * j.g.nt + n / bn) * size + (row % bm) * (nmat * bn) + n % bn;
  floatx4 v[1] = {*reinterpret_cast<const floatx4*>(p)}, u[1] = {{0.f, 0.f, 0.f, 0.f}};
  if (nmat == 2) u[0] = *reinterpret_cast<const floatx4*>(p + bn);
#pragma unroll 4
  for (int q = 1; q < j.S; ++q) {
    v[0] += *reinterpret_cast<const floatx4*>(p + q * tiles * size);
    if (nmat == 2) u[0] += *reinterpret_cast<const floatx4*>(p + q * tiles * size + bn);
  }
  const int64_t row0 = blockIdx.x * 256ll / n4;  // the block's first row
  const Sink sink(j.g.e, row0, 257, j.g.M, j.g.N);
  with_layout(sink, [&](auto vec, auto es) {
    finish<decltype(vec)::value, decltype(es)::value, 1>(sink, (int)(row - row0), 0, n, v, u, load_bias(j.g.e.bias, n, j.g.N),
                                                         load_bias(j.g.e.bias_up, n, j.g.N));
  });
}
__global__ __launch_bounds__(256) void reduce_kernel(Job j, int bm, int bn, int nmat) { reduce_job(j, bm, bn, nmat); }
// All split jobs of a backward pass (blockIdx.y: the job).
__global__ __launch_bounds__(256) void reduce_jobs_kernel(BackwardJobs b, int bm, int bn) {
  reduce_job(b.j[blockIdx.y], bm, bn, 1);
}

__global__ __launch_bounds__(256) void zero_kernel(uint32_t* p, int64_t words) {
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < words; i += gridDim.x * 256ll) p[i] = 0;
}

int round_up(int v, int a) { return (v + a - 1) / a * a; }
int64_t align_up(int64_t v, int64_t a) { return (v + a - 1) / a * a; }

// CUs of the current device (256 if it cannot be asked), looked up once per device.
int device_cus() {
  static std::atomic<int> known[64];
  int dev = 0, cus = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 256;
  cus = known[dev].load(std::memory_order_relaxed);
  if (cus > 0) return cus;
  if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || cus < 1) return 256;
  known[dev].store(cus, std::memory_order_relaxed);
  return cus;
}

void set_tiles(Gemm& g, int kind, int nmat) {
  g.mt = (int)((g.M + kKinds[kind].bm - 1) / kKinds[kind].bm);
  g.nt = (g.N + kKinds[kind].bn / nmat - 1) / (kKinds[kind].bn / nmat);
}

unsigned reduce_blocks(const Job& j) { return (unsigned)((j.g.M * ((j.g.N + 3) / 4) + 255) / 256); }

}  // namespace

size_t linear_ws_bytes(int64_t M, int N, int K, int act) {
  return part_bytes(forward_plan(M, N, K, act == ACT_SWIGLU ? 2 : 1, true, device_cus()).tiles, 1);
}

hipError_t launch_linear(const LinearArgs& a, hipStream_t s) {
  const bool dual = a.act == ACT_SWIGLU;
  const int nmat = dual ? 2 : 1;
  const ForwardPlan f = forward_plan(a.M, a.N, a.K, nmat, a.ws != nullptr, device_cus());
  const int64_t main = a.M - f.rest;
  if (main > 0 && f.tiles.tiles[0] < 1) return hipErrorNotSupported;  // (no tiling has few enough workgroups)
  // The product of rows [row, row + rows).
  auto product = [&](int64_t row, int64_t rows) {
    Gemm g{};
    g.a = {a.x + row * a.K, nullptr, a.K, rows, a.K};
    g.b = {a.w, nullptr, a.K, a.N, a.K};
    g.b_up = {a.w_up, nullptr, a.K, a.N, a.K};
    g.M = rows;
    g.N = a.N;
    g.nk = g.seg = stages(a.K);
    const int64_t at = row * a.N, es = a.out_f32 ? 4 : 2;
    g.e = {a.bias, a.bias_up, a.residual ? static_cast<const char*>(a.residual) + at * es : nullptr,
           static_cast<char*>(a.out) + at * es, a.z ? a.z + at : nullptr, a.z_up ? a.z_up + at : nullptr, a.act, a.out_f32};
    return g;
  };
  hipError_t e = hipSuccess;
  if (f.rest > 0) {
    const Gemm g = product(main, f.rest);
    if (dual) hipLaunchKernelGGL((skinny_kernel<true, 8, 2>), dim3((a.N + 7) / 8), dim3(512), 0, s, g);
    else hipLaunchKernelGGL((skinny_kernel<false, 8, 2>), dim3((a.N + 15) / 16), dim3(512), 0, s, g);
    e = hipGetLastError();
  }
  if (main == 0 || e != hipSuccess) return e;
  const Plan& p = f.tiles;
  Job j{};
  j.g = product(0, main);
  set_tiles(j.g, p.kind, nmat);
  j.S = p.S[0];
  j.part = static_cast<float*>(a.ws);
  const dim3 grid((unsigned)(p.tiles[0] * j.S)), block(kKinds[p.kind].threads());
#define MOE_FORWARD(KIND_)                                                             \
  do {                                                                                 \
    if (dual) hipLaunchKernelGGL((forward_kernel<KIND_, 2>), grid, block, 0, s, j);    \
    else hipLaunchKernelGGL((forward_kernel<KIND_, 1>), grid, block, 0, s, j);         \
  } while (0)
  if (p.kind == 0) MOE_FORWARD(0);
  else if (p.kind == 1) MOE_FORWARD(1);
  else if (p.kind == 2) MOE_FORWARD(2);
  else MOE_FORWARD(3);
#undef MOE_FORWARD
  e = hipGetLastError();
  if (e == hipSuccess && j.S > 1) {
    hipLaunchKernelGGL(reduce_kernel, dim3(reduce_blocks(j)), dim3(256), 0, s, j, kKinds[p.kind].bm,
                       kKinds[p.kind].bn / nmat, nmat);
    e = hipGetLastError();
  }
  return e;
}

// Workspace of the backward pass: dz [M, ld] bf16, the bias gradients' block sums, the split products' sums.
struct BackwardLayout {
  int mats, Np, ld;
  int64_t blocks;  // row blocks of dz_kernel
  size_t sums, parts, total;
  Plan plan;
};

// Products in the order of the plan: the weight gradients, then the input gradient.
static BackwardLayout backward_layout(int64_t M, int N, int K, int act) {
  BackwardLayout l{};
  l.mats = act == ACT_SWIGLU ? 2 : 1;
  l.Np = round_up(N, BK);
  l.ld = l.mats * l.Np;
  l.blocks = (M + kDzRows - 1) / kDzRows;
  l.sums = (size_t)align_up(M * l.ld * 2, 256);
  l.parts = l.sums + (size_t)align_up(l.blocks * l.mats * N * 4, 256);
  Size z[3];
  for (int m = 0; m < l.mats; ++m) z[m] = {N, K, stages(M)};
  z[l.mats] = {M, K, l.mats * stages(N)};
  l.plan = make_plan(z, l.mats + 1, 1, true, device_cus());
  l.total = l.parts + part_bytes(l.plan, l.mats + 1);
  return l;
}

size_t linear_backward_ws_bytes(int64_t M, int N, int K, int act) {
  return M == 0 ? 0 : backward_layout(M, N, K, act).total;
}

hipError_t launch_linear_backward(const LinearBwdArgs& a, hipStream_t s) {
  if (a.M == 0) {
    const int64_t n = (int64_t)a.N * a.K / 2;  // words of a weight gradient (K % 8 == 0)
    struct { void* p; int64_t words; } z[] = {{a.d_w, n}, {a.d_w_up, n}, {a.d_bias, a.N}, {a.d_bias_up, a.N}};
    hipError_t e = hipSuccess;
    for (auto& o : z)
      if (o.p) {
        hipLaunchKernelGGL(zero_kernel, dim3(256), dim3(256), 0, s, static_cast<uint32_t*>(o.p), o.words);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
      }
    return e;
  }
  const BackwardLayout l = backward_layout(a.M, a.N, a.K, a.act);
  if (l.plan.tiles[0] < 1) return hipErrorNotSupported;  // (no tiling has few enough workgroups)
  const int mats = l.mats, Np = l.Np, ld = l.ld;
  uint16_t* dz = static_cast<uint16_t*>(a.ws);
  float* sums = reinterpret_cast<float*>(static_cast<char*>(a.ws) + l.sums);
  char* parts = static_cast<char*>(a.ws) + l.parts;
  const bool bias = a.d_bias || a.d_bias_up;
  constexpr int64_t kMaxBlocks = 65535;  // row blocks per launch
  for (int64_t b = 0; b < l.blocks; b += kMaxBlocks) {
    const int64_t nb = l.blocks - b < kMaxBlocks ? l.blocks - b : kMaxBlocks, r = b * kDzRows;
    const char* d_out = static_cast<const char*>(a.d_out) + r * a.N * (a.out_f32 ? 4 : 2);
    const uint16_t *z = a.z ? a.z + r * a.N : nullptr, *z_up = a.z_up ? a.z_up + r * a.N : nullptr;
    float* part = bias ? sums + b * mats * a.N : nullptr;
    if (a.N % 8 == 0)
      hipLaunchKernelGGL(dz_kernel<8>, dim3((Np + 511) / 512, (unsigned)nb), dim3(256), 0, s, d_out, a.out_f32, z, z_up,
                         a.act, a.M - r, a.N, Np, ld, dz + r * ld, part);
    else
      hipLaunchKernelGGL(dz_kernel<1>, dim3((Np + 63) / 64, (unsigned)nb), dim3(256), 0, s, d_out, a.out_f32, z, z_up,
                         a.act, a.M - r, a.N, Np, ld, dz + r * ld, part);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }

  BackwardJobs jobs{};
  int64_t blocks = 0;
  auto add = [&](const Gemm& g, int q) {  // product q of the plan
    Job& j = jobs.j[jobs.n++];
    j.g = g;
    j.g.e.act = ACT_NONE;
    set_tiles(j.g, l.plan.kind, 1);
    j.S = l.plan.S[q];
    j.first = (int)blocks;
    size_t off = 0;
    for (int i = 0; i < q; ++i) off += l.plan.part_bytes[i];
    j.part = reinterpret_cast<float*>(parts + off);
    blocks += l.plan.tiles[q] * j.S;
  };
  if (a.d_x) {
    Gemm g{};
    g.a = {dz, nullptr, ld, a.M, ld};
    g.b = {a.w, a.w_up, a.K, a.K, a.N};
    g.M = a.M;
    g.N = a.K;
    g.seg = stages(a.N);
    g.nk = mats * g.seg;
    g.e.out = a.d_x;
    add(g, mats);
  }
  jobs.nx = jobs.n;
  for (int m = 0; m < mats; ++m) {
    uint16_t* d_w = m ? a.d_w_up : a.d_w;
    if (!d_w) continue;
    Gemm g{};
    g.a = {dz + m * Np, nullptr, ld, Np, a.M};
    g.b = {a.x, nullptr, a.K, a.K, a.M};
    g.M = a.N;
    g.N = a.K;
    g.nk = g.seg = stages(a.M);
    g.e.out = d_w;
    add(g, m);
  }
  jobs.bias_first = (int)blocks;
  jobs.bias = {sums, l.blocks, a.N, mats, a.d_bias, a.d_bias_up};
  if (bias) blocks += (mats * (int64_t)a.N + 63) / 64;
  if (blocks == 0) return hipSuccess;
  const Kind& kind = kKinds[l.plan.kind];
  const dim3 grid((unsigned)blocks), block(kind.threads());
  if (l.plan.kind == 0) hipLaunchKernelGGL(backward_kernel<0>, grid, block, 0, s, jobs);
  else if (l.plan.kind == 1) hipLaunchKernelGGL(backward_kernel<1>, grid, block, 0, s, jobs);
  else if (l.plan.kind == 2) hipLaunchKernelGGL(backward_kernel<2>, grid, block, 0, s, jobs);
  else hipLaunchKernelGGL(backward_kernel<3>, grid, block, 0, s, jobs);
  hipError_t e = hipGetLastError();
  unsigned most = 0;
  for (int q = 0; q < jobs.n; ++q)
    if (jobs.j[q].S > 1 && reduce_blocks(jobs.j[q]) > most) most = reduce_blocks(jobs.j[q]);
  if (e == hipSuccess && most > 0) {
    hipLaunchKernelGGL(reduce_jobs_kernel, dim3(most, jobs.n), dim3(256), 0, s, jobs, kind.bm, kind.bn);
    e = hipGetLastError();
  }
  return e;
}

}  // namespace moe
