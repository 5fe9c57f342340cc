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
#include "operators.h"

#include <type_traits>

namespace moe {
namespace {

constexpr int BK = 64;  // reduction indices per stage

typedef __attribute__((__vector_size__(4 * sizeof(uint32_t)))) uint32_t u32x4;
typedef __attribute__((__vector_size__(4 * sizeof(short)))) short s16x4;

__device__ __forceinline__ float bf2f(uint16_t h) { return __builtin_bit_cast(float, (uint32_t)h << 16); }

// Raw buffer resource over [base, base + bytes): out-of-range reads return zero.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* base, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, 0x00020000);
}
constexpr uint32_t kOut = 0x80000000u;  // a byte offset past every resource

// 1 / (1 + e^-z) with the hardware exp2 and reciprocal (about 1 ulp each).
__device__ __forceinline__ float sigmoid_f(float z) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-z * 1.4426950408889634f));
}

// act(z) (SwiGLU: silu(z), to be multiplied by u).
__device__ __forceinline__ float activate(int act, float z) {
  switch (act) {
    case ACT_GELU: return 0.5f * z * (1.0f + erff(z * 0.70710678118654752f));
    case ACT_NONE: return z;
    default: return z * sigmoid_f(z);
  }
}
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
// Rows operand: LDS row of 128 B per operand row, 16-byte chunk index XORed with row / 2.  A fragment read takes 16
// rows at four chunks; the 16 lanes served together are rows 0-3 and 12-15 at one chunk and rows 4-11 at the next
// one (or the other way round), which this spreads over all 64 banks, as it does 16 rows at one chunk.
__device__ __forceinline__ int swz(int row) { return (row >> 1) & 7; }
// Columns operand of C columns: LDS row of 2 C bytes per reduction index; half a wavefront of a transposing read
// takes 32 bytes of each of the rows r..r + 3 and r + 8..r + 11, so the 64-byte unit is XORed with the row and the
// 32-byte half of it with row / 8 to spread those over all 64 banks.
template <int C>
__device__ __forceinline__ int swz_t(int r) {
  return (C >= 128 ? (r & 3) << 2 : ((r >> 1) & 1) << 2) | ((r >> 3) & 1) << 1;
}

// MFMA fragment (16 operand rows from row c0, 32 reduction indices from 32 ks) of a staged operand: lane holds
// row c0 + lane % 16, reduction indices 32 ks + 8 (lane / 16) + 0..7.
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

__device__ __forceinline__ uint2 pack4(floatx4 x) {
  return uint2{(uint32_t)f2bf_bits(x[0]) | ((uint32_t)f2bf_bits(x[1]) << 16),
               (uint32_t)f2bf_bits(x[2]) | ((uint32_t)f2bf_bits(x[3]) << 16)};
}

// The epilogue of NV rows, row0 + r * step, in the four columns from n (a multiple of 4, n < N): g and u hold the
// products.  All of the rows' residuals are loaded before the first store, so NV rows are in flight.
template <int NV>
__device__ __forceinline__ void finish(const Epilogue& e, int64_t row0, int step, int64_t M, int n, int N,
                                       floatx4 (&g)[NV], floatx4 (&u)[NV], floatx4 bias, floatx4 bias_up) {
  const int cnt = N - n < 4 ? N - n : 4;
  const bool vec = (N & 3) == 0;  // then a row's groups of four are aligned
  floatx4 res[NV];
#pragma unroll
  for (int r = 0; r < NV; ++r) {
    const int64_t row = row0 + r * step, at = row * N + n;
    res[r] = floatx4{0.f, 0.f, 0.f, 0.f};
    if (e.residual && row < M) {
      if (e.f32) {
        const float* p = static_cast<const float*>(e.residual) + at;
        if (vec) res[r] = *reinterpret_cast<const floatx4*>(p);
        else
          for (int q = 0; q < cnt; ++q) res[r][q] = p[q];
      } else {
        const uint16_t* p = static_cast<const uint16_t*>(e.residual) + at;
        if (vec) {
          const uint2 h = *reinterpret_cast<const uint2*>(p);
          res[r] = floatx4{bf2f((uint16_t)h.x), bf2f((uint16_t)(h.x >> 16)), bf2f((uint16_t)h.y), bf2f((uint16_t)(h.y >> 16))};
        } else {
          for (int q = 0; q < cnt; ++q) res[r][q] = bf2f(p[q]);
        }
      }
    }
  }
  auto put = [&](uint16_t* o, floatx4 x, int64_t at) {
    const uint2 h = pack4(x);
    if (vec) *reinterpret_cast<uint2*>(o + at) = h;
    else
      for (int q = 0; q < cnt; ++q) o[at + q] = (uint16_t)((q & 2 ? h.y : h.x) >> (16 * (q & 1)));
  };
#pragma unroll
  for (int r = 0; r < NV; ++r) {
    g[r] += bias;
    u[r] += bias_up;
    const int64_t row = row0 + r * step;
    if (row < M) {
      if (e.z) put(e.z, g[r], row * N + n);
      if (e.z_up) put(e.z_up, u[r], row * N + n);
    }
  }
  activate_all<NV>(e.act, g, u);
#pragma unroll
  for (int r = 0; r < NV; ++r) {
    const int64_t row = row0 + r * step, at = row * N + n;
    const floatx4 v = g[r] + res[r];
    if (row >= M) continue;
    if (!e.f32) {
      put(static_cast<uint16_t*>(e.out), v, at);
    } else {
      float* o = static_cast<float*>(e.out) + at;
      if (vec) *reinterpret_cast<floatx4*>(o) = v;
      else
        for (int q = 0; q < cnt; ++q) o[q] = v[q];
    }
  }
}

// Four consecutive biases from column n, zeros past N or where there is none.
__device__ __forceinline__ floatx4 load_bias(const float* b, int n, int N) {
  floatx4 v = {0.f, 0.f, 0.f, 0.f};
  if (b)
    for (int q = 0; q < 4; ++q)
      if (n + q < N) v[q] = b[n + q];
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

// One BM x BN output tile per workgroup (NMAT = 2: BN columns of both matrices), NW wavefronts in 2 x NW / 2.
//
// Two LDS buffers and register-staged loads: while stage kt is computed from one buffer, stage kt + 1 goes from
// registers into the other and the registers reload with stage kt + 2.  A stage is four phases, the two halves of
// the wave tile's rows at each of the two 32-wide steps; each phase's fragments are read during the phase before,
// and LDS writes and loads are spread over the MFMAs of the first three.  All of a stage's fragments have been read
// when its last phase begins: there the workgroup synchronises, and the last phase reads the next stage's first
// fragments.  Stages past the end load through a resource of no bytes, so every iteration is the same.
template <int BM, int BN, bool A_COLS, bool B_COLS, int NMAT, int NW>
struct Tile {
  static constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128;
  static constexpr int STAGE = A_BYTES + NMAT * B_BYTES;
  static constexpr int WT_M = BM / 2, WT_N = BN / (NW / 2);         // wave tile (per matrix)
  static constexpr int TM = WT_M / 16, TN = WT_N / 16;
  static constexpr int HM = TM / 2, NB = NMAT * TN;                // fragments of half the rows; of the columns
  static constexpr int A_PIECES = BM / (8 * NW), B_PIECES = BN / (8 * NW);  // loads per wavefront and stage
  static constexpr int WP = NMAT * B_PIECES, LOADS = A_PIECES + WP;
  static constexpr int NMFMA = HM * NB;                             // per phase
  static constexpr int PS = (LOADS + 2) / 3;                        // pieces per phase
  static constexpr int PITCH = NMAT * BN + 4;                       // floats per row of the staged result
  static constexpr int SMEM = 2 * STAGE > 64 * PITCH * 4 ? 2 * STAGE : 64 * PITCH * 4;
  static_assert(HM >= 1 && TN >= 1 && A_PIECES >= 1 && B_PIECES >= 1, "tile too small for the wavefronts");

  // An operand's C rows (columns) from c0 on, as this lane loads them.  Stage kt is read through a resource based
  // at its first element; rows and reduction indices past the operand's end lie outside of it.
  template <bool COLS, int C>
  struct Source {
    const char *base, *base2;  // stage 0 of the two segments (base2 less the first segment's stages)
    int64_t adv;               // bytes between stages
    int full, tail;            // resource bytes of a stage, and of a segment's last stage
    int seg, k1;
    uint32_t off, step;        // this lane's byte offset of piece 0, and between pieces
    int klim;                  // rows operand: stages whose chunk of this lane lies before the reduction's end

    __device__ __forceinline__ Source(const Operand& o, int64_t c0, int seg_, int k1_, int wave, int lane)
        : seg(seg_), k1(k1_) {
      adv = COLS ? BK * o.ld * 2 : BK * 2;
      base = reinterpret_cast<const char*>(o.p + (COLS ? c0 : c0 * o.ld));
      base2 = o.p2 ? reinterpret_cast<const char*>(o.p2 + (COLS ? c0 : c0 * o.ld)) - seg * adv : nullptr;
      if (!COLS) {
        const int left = (int)(o.extent - c0 < C ? o.extent - c0 : C);
        full = tail = (int)(((left - 1) * o.ld + BK) * 2);
        const int row = wave * 8 + (lane >> 3), chunk = (lane & 7) ^ swz(row);
        off = (uint32_t)((row * o.ld + chunk * 8) * 2);
        step = (uint32_t)(8 * NW * o.ld * 2);
        klim = (int)((o.R - chunk * 8 + BK - 1) / BK);
      } else {
        constexpr int LPR = C / 8;  // lanes per LDS row
        const int last = (int)(o.R - (int64_t)(seg - 1) * BK);  // reduction indices in a segment's last stage
        full = (int)(((BK - 1) * o.ld + (o.extent - c0)) * 2);
        tail = (int)(((last - 1) * o.ld + (o.extent - c0)) * 2);
        const int r = wave * (64 / LPR) + lane / LPR, chunk = (lane % LPR) ^ swz_t<C>(r);
        off = c0 + chunk * 8 < o.extent ? (uint32_t)((r * o.ld + chunk * 8) * 2) : kOut;
        step = (uint32_t)(NW * (64 / LPR) * o.ld * 2);
        klim = 0;
      }
    }
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(int kt) const {
      const bool second = base2 && kt >= seg;
      const bool short_stage = COLS && (kt == seg - 1 || kt == 2 * seg - 1);
      const int bytes = kt >= k1 ? 0 : short_stage ? tail : full;
      return make_rsrc((second ? base2 : base) + kt * adv, bytes);
    }
    __device__ __forceinline__ uint32_t offset(int kt) const { return COLS || kt < klim ? off : kOut; }
  };

  struct Stage {  // where a stage's loads come from
    __amdgpu_buffer_rsrc_t a, b, bu;
    uint32_t oa, ob;
  };

  static __device__ __forceinline__ void run(char* smem, const Gemm& g, int64_t m0, int n0, int k0, int k1,
                                             float* part) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / (NW / 2), wn = wave % (NW / 2);
    const Source<A_COLS, BM> src_a(g.a, m0, A_COLS ? g.seg : g.nk, k1, wave, lane);
    const Source<B_COLS, BN> src_b(g.b, n0, g.seg, k1, wave, lane);
    const Source<B_COLS, BN> src_u(NMAT == 2 ? g.b_up : g.b, n0, g.seg, k1, wave, lane);
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

    // Epilogue: 32 rows of either half at a time through LDS, so that global memory is accessed along rows.  The
    // columns' side feeds the MFMA's rows, so a lane holds, for row lane % 16 of a 16-row block, columns
    // 4 (lane / 16) + 0..3 of a 16-column block.
    float* sm = reinterpret_cast<float*>(smem);
    constexpr int C4 = BN / 4, STEP = NW * 64 / C4, NV = 32 / STEP < 4 ? 32 / STEP : 4;  // a thread keeps its columns
    const int n = (threadIdx.x % C4) * 4;
    const floatx4 bias = load_bias(g.e.bias, n0 + n, g.N), bias_up = load_bias(g.e.bias_up, n0 + n, g.N);
#pragma unroll 1
    for (int i = 0; i < TM / 2; ++i) {
      __syncthreads();
#pragma unroll
      for (int ii = 0; ii < TM / 2; ++ii) {
        if (ii != i) continue;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < NB; ++j) {
            const int c = (j / TN) * BN + wn * WT_N + (j % TN) * 16 + (lane >> 4) * 4;
            *reinterpret_cast<floatx4*>(sm + (wm * 32 + h * 16 + (lane & 15)) * PITCH + c) = acc[j][2 * ii + h];
          }
      }
      __syncthreads();
      if (n0 + n >= g.N) continue;
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {  // the 32 rows of the upper and lower half of the tile
        const int64_t row0 = m0 + h * (BM / 2) + i * 32;
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
          if (part) {
#pragma unroll
            for (int r = 0; r < NV; ++r) {
              float* o = part + (int64_t)(h * (BM / 2) + i * 32 + rt + r * STEP) * (NMAT * BN) + n;
              *reinterpret_cast<floatx4*>(o) = v[r];
              if (NMAT == 2) *reinterpret_cast<floatx4*>(o + BN) = u[r];
            }
          } else {
            finish<NV>(g.e, row0 + rt, STEP, g.M, n0 + n, g.N, v, u, bias, bias_up);
          }
        }
      }
    }
  }
};

constexpr int kXcds = 8;
constexpr int kGroupM = 8;  // row tiles per rasterisation group

// Workgroup -> tile: workgroups go round-robin to the XCDs, and each XCD's run of tiles is contiguous in an order
// of groups of kGroupM row tiles, column by column, so that tiles that run together share operand panels in its L2.
__device__ __forceinline__ void tile_of(int bid, int G, int mt, int nt, int& ti, int& tj) {
  const int q = G / kXcds, r = G % kXcds, x = bid % kXcds;
  const int vid = x * q + (x < r ? x : r) + bid / kXcds;
  const int per = kGroupM * nt, grp = vid / per, rem = vid % per;
  const int rows = mt - grp * kGroupM < kGroupM ? mt - grp * kGroupM : kGroupM;
  tj = rem / rows;
  ti = grp * kGroupM + rem % rows;
}

// 256-row tiles: 8 wavefronts, two per SIMD; 128-row tiles: 4, and two workgroups per CU.
constexpr int waves(int BM) { return BM == 256 ? 8 : 4; }

template <int BM, int BN, bool A_COLS, bool B_COLS, int NMAT>
__global__ __launch_bounds__(waves(BM) * 64, 2) void gemm_kernel(Gemm g) {
  using T = Tile<BM, BN, A_COLS, B_COLS, NMAT, waves(BM)>;
  __shared__ __attribute__((aligned(1024))) char smem[T::SMEM];
  int ti, tj;
  tile_of(blockIdx.x, gridDim.x, g.mt, g.nt, ti, tj);
  T::run(smem, g, (int64_t)ti * BM, tj * BN, 0, g.nk, nullptr);
}

// ---------------------------------------------------------------------------
// dz, and the bias gradients
// ---------------------------------------------------------------------------
constexpr int kDzRows = 64;  // rows per block of dz_kernel

// dz (SwiGLU: dz and dz_up, dz_up at column offset Np) rounded to bf16, [M, ld] with zeros in columns
// [N, Np) of each, and the block's column sums of the unrounded values, part[block row][mats][N].
__global__ __launch_bounds__(256) void dz_kernel(const void* __restrict__ d_out, bool f32,
                                                 const uint16_t* __restrict__ z, const uint16_t* __restrict__ z_up,
                                                 int act, int64_t M, int N, int Np, int ld, uint16_t* __restrict__ dz,
                                                 float* __restrict__ part) {
  const int n = blockIdx.x * 256 + threadIdx.x;
  if (n >= Np) return;
  const int64_t r0 = (int64_t)blockIdx.y * kDzRows, r1 = r0 + kDzRows < M ? r0 + kDzRows : M;
  const bool dual = act == ACT_SWIGLU;
  float s0 = 0.f, s1 = 0.f;
  for (int64_t r = r0; r < r1; ++r) {
    float d = 0.f, du = 0.f;
    if (n < N) {
      const int64_t at = r * N + n;
      const float go = f32 ? static_cast<const float*>(d_out)[at] : bf2f(static_cast<const uint16_t*>(d_out)[at]);
      if (act == ACT_NONE) {
        d = go;
      } else {
        const float zz = bf2f(z[at]);
        d = go * activate_grad(act, zz);
        if (dual) {
          d *= bf2f(z_up[at]);
          du = go * activate(act, zz);
        }
      }
    }
    dz[r * ld + n] = f2bf_bits(d);
    if (dual) dz[r * ld + Np + n] = f2bf_bits(du);
    s0 += d;
    s1 += du;
  }
  if (part && n < N) {
    float* p = part + (int64_t)blockIdx.y * (dual ? 2 : 1) * N;
    p[n] = s0;
    if (dual) p[N + n] = s1;
  }
}

// Sums the blocks' column sums in order.
__global__ __launch_bounds__(256) void bias_sum_kernel(const float* __restrict__ part, int64_t blocks, int N, int mats,
                                                       float* __restrict__ d_bias, float* __restrict__ d_bias_up) {
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= mats * N) return;
  float s = 0.f;
  for (int64_t b = 0; b < blocks; ++b) s += part[b * mats * N + c];
  float* o = c < N ? d_bias : d_bias_up;
  if (o) o[c < N ? c : c - N] = s;
}

__global__ __launch_bounds__(256) void zero_kernel(uint32_t* p, int64_t words) {
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < words; i += gridDim.x * 256ll) p[i] = 0;
}

int round_up(int v, int a) { return (v + a - 1) / a * a; }
int64_t align_up(int64_t v, int64_t a) { return (v + a - 1) / a * a; }

template <int BM, int BN, bool A_COLS, bool B_COLS, int NMAT>
hipError_t run_gemm(Gemm g, hipStream_t s) {
  const int64_t mt = (g.M + BM - 1) / BM, nt = (g.N + BN - 1) / BN;
  if (mt * nt > INT32_MAX) return hipErrorInvalidValue;
  g.mt = (int)mt;
  g.nt = (int)nt;
  hipLaunchKernelGGL((gemm_kernel<BM, BN, A_COLS, B_COLS, NMAT>), dim3((unsigned)(mt * nt)), dim3(waves(BM) * 64), 0, s, g);
  return hipGetLastError();
}

int stages(int64_t R) { return (int)((R + BK - 1) / BK); }

}  // namespace

size_t linear_ws_bytes(int64_t, int, int, int) { return 0; }

hipError_t launch_linear(const LinearArgs& a, hipStream_t s) {
  Gemm g{};
  g.a = {a.x, nullptr, a.K, a.M, a.K};
  g.b = {a.w, nullptr, a.K, a.N, a.K};
  g.b_up = {a.w_up, nullptr, a.K, a.N, a.K};
  g.M = a.M;
  g.N = a.N;
  g.nk = g.seg = stages(a.K);
  g.e = {a.bias, a.bias_up, a.residual, a.out, a.z, a.z_up, a.act, a.out_f32};
  const bool big = a.M >= 1024 && a.N >= 1024;
  if (a.act == ACT_SWIGLU) return big ? run_gemm<256, 128, false, false, 2>(g, s) : run_gemm<128, 64, false, false, 2>(g, s);
  return big ? run_gemm<256, 256, false, false, 1>(g, s) : run_gemm<128, 128, false, false, 1>(g, s);
}

// Workspace of the backward pass: dz [M, ld] bf16, then the bias gradients' block sums.
size_t linear_backward_ws_bytes(int64_t M, int N, int K, int act) {
  const int mats = act == ACT_SWIGLU ? 2 : 1;
  const int64_t ld = (int64_t)mats * round_up(N, BK);
  return (size_t)(align_up(M * ld * 2, 256) + align_up((M + kDzRows - 1) / kDzRows * mats * N * 4, 256));
}

hipError_t launch_linear_backward(const LinearBwdArgs& a, hipStream_t s) {
  const int mats = a.act == ACT_SWIGLU ? 2 : 1;
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
  const int Np = round_up(a.N, BK), ld = mats * Np;
  uint16_t* dz = static_cast<uint16_t*>(a.ws);
  float* part = reinterpret_cast<float*>(static_cast<char*>(a.ws) + align_up(a.M * ld * 2, 256));
  const int64_t blocks = (a.M + kDzRows - 1) / kDzRows;
  const bool sums = a.d_bias || a.d_bias_up;
  // At most 65535 block rows per launch.
  constexpr int64_t kMaxBlocks = 65535;
  for (int64_t b = 0; b < blocks; b += kMaxBlocks) {
    const int64_t nb = blocks - b < kMaxBlocks ? blocks - b : kMaxBlocks, r = b * kDzRows;
    const int64_t rows = a.M - r;
    const char* d_out = static_cast<const char*>(a.d_out) + r * a.N * (a.out_f32 ? 4 : 2);
    hipLaunchKernelGGL(dz_kernel, dim3((Np + 255) / 256, (unsigned)nb), dim3(256), 0, s, d_out, a.out_f32,
                       a.z ? a.z + r * a.N : nullptr, a.z_up ? a.z_up + r * a.N : nullptr, a.act, rows, a.N, Np, ld,
                       dz + r * ld, sums ? part + b * mats * a.N : nullptr);
  }
  if (sums)
    hipLaunchKernelGGL(bias_sum_kernel, dim3((mats * a.N + 255) / 256), dim3(256), 0, s, part, blocks, a.N, mats,
                       a.d_bias, a.d_bias_up);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  Gemm g{};
  g.e.act = ACT_NONE;
  if (a.d_x) {
    g.a = {dz, nullptr, ld, a.M, ld};
    g.b = {a.w, a.w_up, a.K, a.K, a.N};
    g.M = a.M;
    g.N = a.K;
    g.seg = stages(a.N);
    g.nk = mats * g.seg;
    g.e.out = a.d_x;
    const bool big = a.M >= 1024 && a.K >= 1024;
    e = big ? run_gemm<256, 256, false, true, 1>(g, s) : run_gemm<128, 128, false, true, 1>(g, s);
    if (e != hipSuccess) return e;
  }
  for (int m = 0; m < mats; ++m) {
    uint16_t* d_w = m ? a.d_w_up : a.d_w;
    if (!d_w) continue;
    g.a = {dz + m * Np, nullptr, ld, Np, a.M};
    g.b = {a.x, nullptr, a.K, a.K, a.M};
    g.M = a.N;
    g.N = a.K;
    g.nk = g.seg = stages(a.M);
    g.e.out = d_w;
    const bool big = a.N >= 1024 && a.K >= 1024;
    e = big ? run_gemm<256, 256, true, true, 1>(g, s) : run_gemm<128, 128, true, true, 1>(g, s);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace moe
