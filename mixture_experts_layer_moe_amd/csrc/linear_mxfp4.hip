// Products of MXFP4 operands, dense and grouped by expert, with bias, activation and residual in the epilogue.
//
//   z[m, n] = sum over k of x[m, k] w[n, k] + bias[n];  out = act(z) [* z_up] + residual
//
// Both operands have k contiguous, two codes a byte, and a scale byte per 32 values, which is what the scaled matrix
// instructions take: v_mfma_scale_f32_32x32x64_f8f6f4 (16x16x128) multiplies 32 codes a lane, one block, whose scale is
// one byte of a register.  The products of two codes and their scales are exact, sums are fp32.
//
// The weights feed the instruction's rows and the tokens its columns, so that a lane's results belong to one token.
#include "activation.h"

#include <type_traits>

namespace moe {
namespace {

typedef __attribute__((__vector_size__(16 * sizeof(float)))) float floatx16;
typedef __attribute__((__vector_size__(8 * sizeof(int)))) int intx8;
typedef __attribute__((address_space(3))) void lds_void;

constexpr uint32_t kOut = 0x80000000u;  // a byte offset past every resource
constexpr int kStage = 256;             // reduction indices per stage of a tile: 128 bytes a row
constexpr int kFp4 = 4;                 // the matrix instructions' operand format

// s_waitcnt vmcnt(n), other counters left alone.
template <int n>
__device__ __forceinline__ void wait_vmcnt() {
  __builtin_amdgcn_s_waitcnt((n & 15) | (7 << 4) | (15 << 8) | ((n >> 4) << 14));
}
__device__ __forceinline__ void wait_lgkm0() { __builtin_amdgcn_s_waitcnt(15 | (7 << 4) | (0 << 8) | (3 << 14)); }
__device__ __forceinline__ void ring_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

__device__ __forceinline__ intx8 widen(u32x4 v) { return intx8{(int)v[0], (int)v[1], (int)v[2], (int)v[3], 0, 0, 0, 0}; }

// Which rows and weights a tile has.
struct Rows {
  int64_t row0;  // first row of out (and of x, unless gathered)
  int valid;     // rows that exist, <= 0: none
  int expert;
};

struct Product {
  MxLinearArgs a;
  int mt, nt;  // tiles (grouped: mt is the capacity's)
  int sub;     // row tiles of a permutation tile
};

template <bool GROUPED>
__device__ __forceinline__ Rows rows_of(const Product& p, int ti, int bm) {
  Rows r;
  if constexpr (GROUPED) {
    const int t = ti / p.sub;
    r.expert = p.a.tiles[2 * t];
    const int first = p.a.tiles[2 * t + 1] + (ti - t * p.sub) * bm;
    r.row0 = first;
    r.valid = p.a.offsets[r.expert] + p.a.counts[r.expert] - first;
  } else {
    r.expert = 0;
    r.row0 = (int64_t)ti * bm;
    const int64_t left = p.a.M - r.row0;
    r.valid = left < bm ? (int)left : bm;
  }
  if (r.valid > bm) r.valid = bm;
  return r;
}

// ---------------------------------------------------------------------------
// Epilogue
// ---------------------------------------------------------------------------
template <int V>
__device__ __forceinline__ void load_bias(const float* b, int left, bool whole, float (&v)[V]) {
  if (whole) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const floatx4 q = *reinterpret_cast<const floatx4*>(b + i);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[i + e] = q[e];
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < left) v[i] = b[i];
  }
}

// V values of one row from column n: bias, activation, residual, rounding, stores.  `at` is the element's index in out.
template <int V>
__device__ __forceinline__ void finish(const MxLinearArgs& a, int64_t at, int n, float (&z)[V], const float (&u)[V]) {
  constexpr int W = V < 8 ? V : 8;  // bf16 values per access
  const int left = a.N - n;         // columns that exist
  if (left <= 0) return;
  const bool whole = left >= V && a.N % 8 == 0;  // (then every row's groups of V are 16-byte aligned)
  float bz[V], bu[V];
#pragma unroll
  for (int i = 0; i < V; ++i) bz[i] = bu[i] = 0.f;
  if (a.bias) load_bias<V>(a.bias + n, left, whole, bz);
  if (a.bias_up) load_bias<V>(a.bias_up + n, left, whole, bu);
  switch (a.act) {
    case ACT_NONE:
#pragma unroll
      for (int i = 0; i < V; ++i) z[i] += bz[i];
      break;
    case ACT_GELU:
#pragma unroll
      for (int i = 0; i < V; ++i) z[i] = activate(ACT_GELU, z[i] + bz[i]);
      break;
    case ACT_SILU:
#pragma unroll
      for (int i = 0; i < V; ++i) z[i] = activate(ACT_SILU, z[i] + bz[i]);
      break;
    default:
#pragma unroll
      for (int i = 0; i < V; ++i) z[i] = activate(ACT_SILU, z[i] + bz[i]) * (u[i] + bu[i]);
  }
  if (a.out_f32) {
    float* o = static_cast<float*>(a.out) + at;
    const float* r = static_cast<const float*>(a.residual);
    if (whole) {
#pragma unroll
      for (int i = 0; i < V; i += 4) {
        floatx4 v = {z[i], z[i + 1], z[i + 2], z[i + 3]};
        if (r) v += *reinterpret_cast<const floatx4*>(r + at + i);
        *reinterpret_cast<floatx4*>(o + i) = v;
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i < left) o[i] = r ? z[i] + r[at + i] : z[i];
    }
  } else {
    uint16_t* o = static_cast<uint16_t*>(a.out) + at;
    const uint16_t* r = static_cast<const uint16_t*>(a.residual);
    if (whole) {
      typedef __attribute__((__vector_size__(W * 2))) uint32_t words;  // W values
#pragma unroll
      for (int i = 0; i < V; i += W) {
        words h;
        if (r) {
          const words q = *reinterpret_cast<const words*>(r + at + i);
#pragma unroll
          for (int e = 0; e < W; ++e) z[i + e] += bf2f((uint16_t)(q[e >> 1] >> (16 * (e & 1))));
        }
#pragma unroll
        for (int e = 0; e < W / 2; ++e)
          h[e] = (uint32_t)f2bf_bits(z[i + 2 * e]) | ((uint32_t)f2bf_bits(z[i + 2 * e + 1]) << 16);
        *reinterpret_cast<words*>(o + i) = h;
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i < left) o[i] = f2bf_bits(r ? z[i] + bf2f(r[at + i]) : z[i]);
    }
  }
}

// ---------------------------------------------------------------------------
// Tiles through LDS
// ---------------------------------------------------------------------------
constexpr int kXcds = 8;
constexpr int kGroupM = 8;  // row tiles per rasterisation group

// Workgroup -> tile: workgroups go round-robin to the XCDs; each XCD's run is contiguous in an order of groups of
// kGroupM row tiles, column by column, so that tiles that run together share operand panels in its L2.
__device__ __forceinline__ void tile_of(int bid, int mt, int nt, int& ti, int& tj) {
  const int G = mt * nt, each = G / kXcds, more = G % kXcds, x = bid % kXcds;
  const int vid = x * each + (x < more ? x : more) + bid / kXcds;
  const int per = kGroupM * nt, grp = vid / per, rem = vid % per;
  const int rows = mt - grp * kGroupM < kGroupM ? mt - grp * kGroupM : kGroupM;
  tj = rem / rows;
  ti = grp * kGroupM + rem % rows;
}

// Physical 16-byte chunk of logical chunk c in LDS row r is c ^ swz(r).  The 16 lanes that a 16-byte LDS read serves
// together are lanes 0-3, 12-15, 20-27 or 4-11, 16-19, 28-31 (and 32 on): this spreads a fragment's rows over all
// 64 banks.
__device__ __forceinline__ constexpr int swz(int row) { return (row >> 1) & 7; }

// BM rows by BN columns (NMAT = 2: BN of each matrix), WM x WN wavefronts.
//
// Two LDS buffers and register-staged codes: while a stage of 256 reduction indices (128 bytes a row: whole cache lines)
// is multiplied from one buffer, the next stage goes from registers into the other and the registers reload with the one
// after it.  A stage is four steps, each a matrix instruction of 64 indices per accumulator; a step's fragments are read
// during the step before, and the writes and loads are spread over the first three.  When the last step begins the
// stage has been read: there the workgroup synchronises, and the last step reads the next stage's first fragments.
//
// The scales go straight to LDS for two stages at a time, 16 bytes a row: a row's bytes of one stage would each time be
// an access of their own to the row's cache line, nearly as many as the codes need (340 us instead of 294 at
// 4096 x 14336 x 4096 SwiGLU with 128-wide stages).  Lane half h takes the stage's blocks 4 h .. 4 h + 3, one for each
// step, whose scales are the bytes of the word that it reads.
template <int BM, int BN, int NMAT, int WM, int WN>
struct Tile {
  static constexpr int NW = WM * WN;
  static constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128;
  static constexpr int STAGE = A_BYTES + NMAT * B_BYTES;
  static constexpr int ROWS = BM + NMAT * BN;  // of x, then of the matrices
  static constexpr int SCALES = 2 * STAGE;    // two places of 16 bytes a row
  static constexpr int SMEM = SCALES + 2 * ROWS * 16;
  static constexpr int PITCH = NMAT * BN / WN + 4, EPI = 32 * PITCH * 4;  // floats a staged row, bytes of 32 of them
  static constexpr int WT_M = BM / WM, WT_N = BN / WN;
  static constexpr int TM = WT_M / 32, TN = WT_N / 32, NB = NMAT * TN;
  static constexpr int A_PIECES = BM / (8 * NW), B_PIECES = BN / (8 * NW);
  static constexpr int S_ALL = ROWS / 64, S_PIECES = (S_ALL + NW - 1) / NW;
  static constexpr int LOADS = A_PIECES + NMAT * B_PIECES;
  static_assert(BM % (8 * NW) == 0 && BN % (8 * NW) == 0 && BM % 64 == 0 && BN % 64 == 0, "whole pieces");
  static_assert(TM >= 1 && TN >= 1, "tile");
  static_assert(NW * EPI <= SMEM, "room for the results");

  template <bool GROUPED>
  static __device__ __forceinline__ void run(char* smem, const Product& p, const Rows& rw, int n0) {
    const MxLinearArgs& a = p.a;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN, l32 = lane & 31, half = lane >> 5;
    const int kb = a.K / 2, sb = a.K / 32, nk = (a.K + kStage - 1) / kStage;
    const bool gather = GROUPED && a.row_src != nullptr;
    const int cols = a.N - n0 < BN ? a.N - n0 : BN;

    // Resources: x's rows (gathered: all of x), the tile's weight rows.  Rows past them read zeros.
    const int64_t x0 = gather ? 0 : rw.row0, xr = gather ? a.M : rw.valid;
    const __amdgpu_buffer_rsrc_t rx = make_rsrc(a.x.q + x0 * kb, xr * kb);
    const int64_t w0 = (int64_t)rw.expert * a.N + n0;
    const __amdgpu_buffer_rsrc_t rwq[2] = {make_rsrc(a.w.q + w0 * kb, (int64_t)cols * kb),
                                           make_rsrc((NMAT == 2 ? a.w_up.q : a.w.q) + w0 * kb, (int64_t)cols * kb)};
    // Row r of the tile in x, kOut where there is none.
    auto row_of = [&](int r) -> uint32_t {
      if (r >= rw.valid) return kOut;
      if (!gather) return (uint32_t)r;
      const int src = a.row_src[rw.row0 + r];
      const uint32_t t = (uint32_t)src / (uint32_t)a.topk;
      return src >= 0 && t < a.M ? t : kOut;
    };
    // This lane's offsets.  Codes: rows of 8 lanes, 16 bytes each.  Scales: a row a lane.
    const int r_in = lane >> 3, chunk = (lane & 7) ^ swz(wave * 8 + r_in);
    uint32_t off_a[A_PIECES], off_s[S_PIECES];
    __amdgpu_buffer_rsrc_t rs[S_PIECES];
#pragma unroll
    for (int q = 0; q < A_PIECES; ++q) {
      const uint32_t row = row_of((q * NW + wave) * 8 + r_in);
      off_a[q] = row != kOut ? row * (uint32_t)kb + chunk * 16 : kOut;
    }
    const uint32_t off_b = (uint32_t)((wave * 8 + r_in) * kb + chunk * 16);
#pragma unroll
    for (int q = 0; q < S_PIECES; ++q) {
      const int first = ((q * NW + wave) % S_ALL) * 64;  // (a last piece over is loaded twice)
      if (first < BM) {
        const uint32_t row = row_of(first + lane);
        off_s[q] = row != kOut ? row * (uint32_t)sb : kOut;
        rs[q] = make_rsrc(a.x.s + x0 * sb, xr * sb);
      } else {
        const int c = first - BM, m = NMAT == 2 && c >= BN;
        off_s[q] = (uint32_t)((c - m * BN + lane) * sb);
        rs[q] = make_rsrc((m ? a.w_up.s : a.w.s) + w0 * sb, (int64_t)cols * sb);
      }
    }

    // K is a multiple of 128: where the last stage is half a stage, the later half of each row reads zeros.
    const bool odd = (a.K & 128) != 0;
    const uint32_t cut = chunk >= 4 ? kOut : 0;
    // Stage kt's codes, piece by piece: from global memory to registers, from there to LDS.
    u32x4 stg[LOADS];
    auto load = [&](int q, int kt) {  // (stages past the last load from past the resources)
      const uint32_t none = kt < nk ? (odd && kt == nk - 1 ? cut : 0) : kOut, at = (uint32_t)kt * 128;
      if (q < A_PIECES) stg[q] = __builtin_amdgcn_raw_buffer_load_b128(rx, (off_a[q < A_PIECES ? q : 0] + at) | none, 0, 0);
      else stg[q] = __builtin_amdgcn_raw_buffer_load_b128(rwq[(q - A_PIECES) / B_PIECES],
                                                          (off_b + (q - A_PIECES) % B_PIECES * 8 * NW * kb + at) | none, 0, 0);
    };
    auto write = [&](int q, int kt) {
      const int line = q < A_PIECES ? q * NW : BM / 8 + (q - A_PIECES) / B_PIECES * (BN / 8) + (q - A_PIECES) % B_PIECES * NW;
      *reinterpret_cast<u32x4*>(smem + (kt % 2) * STAGE + (line + wave) * 1024 + lane * 16) = stg[q];
    };
    // The scales of stages kt and kt + 1 (16 bytes may run into the next row's, which no stage uses).
    auto issue_scales = [&](int kt) {
#pragma unroll
      for (int q = 0; q < S_PIECES; ++q)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            rs[q], (lds_void*)(smem + SCALES + (kt / 2 % 2) * (ROWS * 16) + ((q * NW + wave) % S_ALL) * 1024), 16, off_s[q] + kt * 8, 0, 0, 0);
    };

    floatx16 acc[NB][TM];
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[j][i][v] = 0.f;

    struct Frags {
      u32x4 a[TM], b[NB];
    };
    struct Scales {
      int a[TM], b[NB];
    };
    auto read = [&](Frags& f, int kt, int step) {
      const char* st = smem + (kt % 2) * STAGE;
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        const int row = wn * WT_N + (j % TN) * 32 + l32;
        f.b[j] = *reinterpret_cast<const u32x4*>(st + A_BYTES + (j / TN) * B_BYTES + row * 128 + (((half * 4 + step) ^ swz(row)) << 4));
      }
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        const int row = wm * WT_M + i * 32 + l32;
        f.a[i] = *reinterpret_cast<const u32x4*>(st + row * 128 + (((half * 4 + step) ^ swz(row)) << 4));
      }
    };
    auto read_scales = [&](Scales& f, int kt) {
      const char* sc = smem + SCALES + (kt / 2 % 2) * (ROWS * 16) + (kt % 2) * 8 + half * 4;
#pragma unroll
      for (int i = 0; i < TM; ++i) f.a[i] = *reinterpret_cast<const int*>(sc + (wm * WT_M + i * 32 + l32) * 16);
#pragma unroll
      for (int j = 0; j < NB; ++j)
        f.b[j] = *reinterpret_cast<const int*>(sc + (BM + (j / TN) * BN + wn * WT_N + (j % TN) * 32 + l32) * 16);
    };
    auto multiply = [&](auto step, const Frags& f, const Scales& s) {
      constexpr int S = decltype(step)::value;
#pragma unroll
      for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int i = 0; i < TM; ++i)
          acc[j][i] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(widen(f.b[j]), widen(f.a[i]), acc[j][i], kFp4, kFp4, S,
                                                                      s.b[j], S, s.a[i]);
      // (the instructions have no side effects: the use of the accumulators keeps them on this side of the barrier)
#pragma unroll
      for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int i = 0; i < TM; ++i) asm volatile("" : "+v"(acc[j][i]));
    };
    // Instruction order of a step: an LDS read after each matrix instruction while there are any, and the pieces' writes
    // and loads in the places after those.
    auto order = [&](auto reads, auto pieces) {
      constexpr int nr = decltype(reads)::value, np = decltype(pieces)::value, nm = NB * TM;
#pragma unroll
      for (int t = 0; t < nm; ++t) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        if (t < nr) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        if (t + nm < nr) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        if (t >= nm - np) {
          __builtin_amdgcn_sched_group_barrier(0x200, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    using std::integral_constant;
    Frags f[2];
    Scales sc, next;
    issue_scales(0);
#pragma unroll
    for (int q = 0; q < LOADS; ++q) load(q, 0);
#pragma unroll
    for (int q = 0; q < LOADS; ++q) write(q, 0);  // (waits for the scales too, which went ahead)
#pragma unroll
    for (int q = 0; q < LOADS; ++q) load(q, 1);
    wait_lgkm0();
    ring_barrier();
    read(f[0], 0, 0);
    read_scales(next, 0);
    constexpr int P0 = (LOADS + 2) / 3, P1 = 2 * P0 < LOADS ? 2 * P0 : LOADS;
    for (int kt = 0; kt < nk; ++kt) {
      if (kt % 2 == 0 && kt + 2 < nk) issue_scales(kt + 2);
      auto pieces = [&](int from, int to) {
#pragma unroll
        for (int q = 0; q < LOADS; ++q)
          if (q >= from && q < to) {
            write(q, kt + 1);
            load(q, kt + 2);
          }
      };
      sc = next;
      if (odd && kt == nk - 1 && half) {  // (no scales there; the codes are zeros)
#pragma unroll
        for (int i = 0; i < TM; ++i) sc.a[i] = 0;
#pragma unroll
        for (int j = 0; j < NB; ++j) sc.b[j] = 0;
      }
      read(f[1], kt, 1);
      pieces(0, P0);
      multiply(integral_constant<int, 0>{}, f[0], sc);
      order(integral_constant<int, TM + NB>{}, integral_constant<int, P0>{});
      read(f[0], kt, 2);
      pieces(P0, P1);
      multiply(integral_constant<int, 1>{}, f[1], sc);
      order(integral_constant<int, TM + NB>{}, integral_constant<int, P1 - P0>{});
      read(f[1], kt, 3);
      pieces(P1, LOADS);
      multiply(integral_constant<int, 2>{}, f[0], sc);
      order(integral_constant<int, TM + NB>{}, integral_constant<int, LOADS - P1>{});
      wait_lgkm0();    // this wavefront's reads of stage kt and writes of stage kt + 1 are done
      ring_barrier();  // so are all others'
      __builtin_amdgcn_sched_barrier(0);
      read(f[0], kt + 1, 0);
      read_scales(next, kt + 1);
      multiply(integral_constant<int, 3>{}, f[1], sc);
      order(integral_constant<int, 2 * (TM + NB)>{}, integral_constant<int, 0>{});
    }
    ring_barrier();

    // A lane holds, for row l32 of a 32-row block, columns 8 (v / 4) + 4 half + v % 4 of each 32-column block (v: element
    // of the accumulator).  32 rows at a time go through this wavefront's part of LDS, so that stores run along rows.
    float* sm = reinterpret_cast<float*>(smem + wave * EPI);
#pragma unroll 1
    for (int i = 0; i < TM; ++i) {
#pragma unroll
      for (int ii = 0; ii < TM; ++ii) {
        if (ii != i) continue;
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
          for (int v = 0; v < 16; v += 4)
            *reinterpret_cast<floatx4*>(sm + l32 * PITCH + j * 32 + 2 * v + half * 4) =
                floatx4{acc[j][ii][v], acc[j][ii][v + 1], acc[j][ii][v + 2], acc[j][ii][v + 3]};
      }
      const int r0 = wm * WT_M + i * 32;
      if (a.out_f32) store_rows<4>(a, rw, sm, r0, n0 + wn * WT_N, lane);
      else store_rows<8>(a, rw, sm, r0, n0 + wn * WT_N, lane);
    }
  }

  // The epilogue of 32 staged rows from row r0 of the tile: V columns a lane.
  template <int V>
  static __device__ __forceinline__ void store_rows(const MxLinearArgs& a, const Rows& rw, const float* sm, int r0, int n0,
                                                    int lane) {
    constexpr int LPR = WT_N / V, STEP = 64 / LPR;  // lanes a row, rows at a time
    const int c = lane % LPR * V;
#pragma unroll 1
    for (int r = lane / LPR; r < 32; r += STEP) {
      float z[V], u[V];
#pragma unroll
      for (int v = 0; v < V; v += 4) {
        const floatx4 p = *reinterpret_cast<const floatx4*>(sm + r * PITCH + c + v);
        const floatx4 q = NMAT == 2 ? *reinterpret_cast<const floatx4*>(sm + r * PITCH + WT_N + c + v) : p;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          z[v + e] = p[e];
          u[v + e] = q[e];
        }
      }
      if (r0 + r < rw.valid) finish<V>(a, (rw.row0 + r0 + r) * a.N + n0 + c, n0 + c, z, u);
    }
  }
};

template <int BM, int BN, int NMAT, int WM, int WN, bool GROUPED>
__global__ __launch_bounds__(WM* WN * 64) void tile_kernel(Product p) {
  using T = Tile<BM, BN / NMAT, NMAT, WM, WN>;
  __shared__ __attribute__((aligned(1024))) char smem[T::SMEM];
  int mt = p.mt;
  if (GROUPED) {
    const int n = *p.a.num_tiles * p.sub;
    mt = n < mt ? n : mt;
  }
  if ((int)blockIdx.x >= mt * p.nt) return;
  int ti, tj;
  tile_of(blockIdx.x, mt, p.nt, ti, tj);
  const Rows rw = rows_of<GROUPED>(p, ti, BM);
  if (rw.valid <= 0) return;
  T::template run<GROUPED>(smem, p, rw, tj * (BN / NMAT));
}

// ---------------------------------------------------------------------------
// Few rows: the weights stream from global memory into the matrix instructions' registers
// ---------------------------------------------------------------------------
// Up to 16 MB rows by 16 columns a workgroup; its wavefronts take turns at units of 512 reduction indices and add up
// through LDS.  v_mfma_scale_f32_16x16x128: lane l holds block l / 16 of four of row l % 16, so a load of 16 bytes a
// lane is 64 contiguous bytes of each of 16 rows, and a unit's 16 scale bytes of a row come as one load.
constexpr int kStreamWaves = 8;

template <int MB, int NMAT, bool GROUPED>
__global__ __launch_bounds__(kStreamWaves * 64) void stream_kernel(Product p) {
  constexpr int RED = NMAT * MB * 256;  // floats of a wavefront's sums
  __shared__ float red[kStreamWaves * RED];
  const MxLinearArgs& a = p.a;
  const int ti = blockIdx.x / p.nt, n0 = (int)(blockIdx.x % p.nt) * 16;
  if (GROUPED && ti >= *a.num_tiles * p.sub) return;
  const Rows rw = rows_of<GROUPED>(p, ti, 16 * MB);
  if (rw.valid <= 0) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  const int kb = a.K / 2, sb = a.K / 32, units = (a.K + 511) / 512;
  const bool gather = GROUPED && a.row_src != nullptr;
  const int cols = a.N - n0 < 16 ? a.N - n0 : 16;
  const int64_t x0 = gather ? 0 : rw.row0, xr = gather ? a.M : rw.valid;
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(a.x.q + x0 * kb, xr * kb), rxs = make_rsrc(a.x.s + x0 * sb, xr * sb);
  const int64_t w0 = (int64_t)rw.expert * a.N + n0;
  const __amdgpu_buffer_rsrc_t rwq[2] = {make_rsrc(a.w.q + w0 * kb, (int64_t)cols * kb),
                                         make_rsrc((NMAT == 2 ? a.w_up.q : a.w.q) + w0 * kb, (int64_t)cols * kb)};
  const __amdgpu_buffer_rsrc_t rws[2] = {make_rsrc(a.w.s + w0 * sb, (int64_t)cols * sb),
                                         make_rsrc((NMAT == 2 ? a.w_up.s : a.w.s) + w0 * sb, (int64_t)cols * sb)};
  uint32_t ox[MB], oxs[MB];
#pragma unroll
  for (int i = 0; i < MB; ++i) {
    const int r = i * 16 + l16;
    uint32_t row = (uint32_t)r;
    bool in = r < rw.valid;
    if (gather) {
      const int src = in ? a.row_src[rw.row0 + r] : -1;
      row = (uint32_t)src / (uint32_t)a.topk;
      in = src >= 0 && row < a.M;
    }
    ox[i] = in ? row * (uint32_t)kb + g * 16 : kOut;
    oxs[i] = in ? row * (uint32_t)sb : kOut;
  }
  const uint32_t ow = (uint32_t)(l16 * kb + g * 16), ows = (uint32_t)(l16 * sb);

  floatx4 acc[NMAT][MB];
#pragma unroll
  for (int m = 0; m < NMAT; ++m)
#pragma unroll
    for (int i = 0; i < MB; ++i) acc[m][i] = floatx4{0.f, 0.f, 0.f, 0.f};

  for (int u = wave; u < units; u += kStreamWaves) {
    const int steps = (a.K - u * 512) / 128;  // (4 but for the last unit)
    u32x4 w[NMAT][4], ws[NMAT], x[MB][4], xs[MB];
    // (steps past the row's end load from past the resource; the scales of a unit may run into the next row's, which
    // no step uses)
#pragma unroll
    for (int m = 0; m < NMAT; ++m) {
#pragma unroll
      for (int s = 0; s < 4; ++s)
        w[m][s] = __builtin_amdgcn_raw_buffer_load_b128(rwq[m], s < steps ? ow + u * 256 + s * 64 : kOut, 0, 2);
      ws[m] = __builtin_amdgcn_raw_buffer_load_b128(rws[m], ows + u * 16, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < MB; ++i) {
#pragma unroll
      for (int s = 0; s < 4; ++s)
        x[i][s] = __builtin_amdgcn_raw_buffer_load_b128(rx, s < steps ? ox[i] + u * 256 + s * 64 : kOut, 0, 0);
      xs[i] = __builtin_amdgcn_raw_buffer_load_b128(rxs, oxs[i] + u * 16, 0, 0);
    }
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      if (s >= steps) break;
#pragma unroll
      for (int m = 0; m < NMAT; ++m) {
        const int sw = (int)(ws[m][s] >> (8 * g));
#pragma unroll
        for (int i = 0; i < MB; ++i)
          acc[m][i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(widen(w[m][s]), widen(x[i][s]), acc[m][i], kFp4, kFp4, 0,
                                                                       sw, 0, (int)(xs[i][s] >> (8 * g)));
      }
    }
  }
#pragma unroll
  for (int m = 0; m < NMAT; ++m)
#pragma unroll
    for (int i = 0; i < MB; ++i) *reinterpret_cast<floatx4*>(red + wave * RED + (m * MB + i) * 256 + lane * 4) = acc[m][i];
  __syncthreads();
  // Lane l of a partial sum: row l % 16, columns 4 (l / 16) + 0..3.  One wavefront per 16 rows, in the units' order.
  if (wave < MB) {
    float z[4] = {0.f, 0.f, 0.f, 0.f}, v[4] = {0.f, 0.f, 0.f, 0.f};
    for (int q = 0; q < kStreamWaves; ++q) {
      const float* s = red + q * RED + wave * 256 + lane * 4;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        z[e] += s[e];
        if (NMAT == 2) v[e] += s[MB * 256 + e];
      }
    }
    const int r = wave * 16 + l16, n = n0 + g * 4;
    if (r < rw.valid) finish<4>(a, (rw.row0 + r) * a.N + n, n, z, v);
  }
}

hipError_t launch(const Product& p0, bool grouped, hipStream_t s) {
  Product p = p0;
  const bool dual = p.a.act == ACT_SWIGLU;
  const int64_t rows = grouped ? p.a.tile_m : p.a.M;  // rows that share weights
#define MOE_LAUNCH(KERNEL_, BLOCK_)                                                                        \
  do {                                                                                                     \
    const int64_t g = (int64_t)p.mt * p.nt;                                                                \
    if (g > 0x7fffffff / (BLOCK_)) return hipErrorNotSupported;                                            \
    hipLaunchKernelGGL((KERNEL_), dim3((unsigned)g), dim3(BLOCK_), 0, s, p);                               \
    return hipGetLastError();                                                                              \
  } while (0)
#define MOE_TILE(BM_, BN_, WM_, WN_)                                                                       \
  do {                                                                                                     \
    if (grouped && dual) MOE_LAUNCH((tile_kernel<BM_, BN_, 2, WM_, WN_, true>), WM_* WN_ * 64);            \
    if (grouped) MOE_LAUNCH((tile_kernel<BM_, BN_, 1, WM_, WN_, true>), WM_* WN_ * 64);                    \
    if (dual) MOE_LAUNCH((tile_kernel<BM_, BN_, 2, WM_, WN_, false>), WM_* WN_ * 64);                      \
    MOE_LAUNCH((tile_kernel<BM_, BN_, 1, WM_, WN_, false>), WM_* WN_ * 64);                                \
  } while (0)
#define MOE_STREAM(MB_)                                                                                    \
  do {                                                                                                     \
    if (grouped && dual) MOE_LAUNCH((stream_kernel<MB_, 2, true>), kStreamWaves * 64);                     \
    if (grouped) MOE_LAUNCH((stream_kernel<MB_, 1, true>), kStreamWaves * 64);                             \
    if (dual) MOE_LAUNCH((stream_kernel<MB_, 2, false>), kStreamWaves * 64);                               \
    MOE_LAUNCH((stream_kernel<MB_, 1, false>), kStreamWaves * 64);                                         \
  } while (0)
  auto tiles = [&](int bm, int bn) {
    if (grouped) {
      p.sub = p.a.tile_m > bm ? p.a.tile_m / bm : 1;
      p.mt = (int)p.a.tiles_cap * p.sub;
    } else {
      p.sub = 1;
      p.mt = (int)((p.a.M + bm - 1) / bm);
    }
    p.nt = (p.a.N + bn - 1) / bn;
  };
  const int mats = dual ? 2 : 1;
  if (rows <= 64) {
    const int mb = rows <= 16 ? 1 : rows <= 32 ? 2 : 4;
    tiles(16 * mb, 16);
    if (mb == 1) MOE_STREAM(1);
    if (mb == 2) MOE_STREAM(2);
    MOE_STREAM(4);
  }
  tiles(256, 256 / mats);
  if (rows >= 256 && (int64_t)p.mt * p.nt >= 192) MOE_TILE(256, 256, 2, 4);
  tiles(128, 128 / mats);
  MOE_TILE(128, 128, 2, 2);
#undef MOE_LAUNCH
#undef MOE_TILE
#undef MOE_STREAM
}

}  // namespace

size_t linear_mxfp4_ws_bytes(int64_t, int, int, int) { return 0; }

hipError_t launch_linear_mxfp4(const MxLinearArgs& a, hipStream_t s) { return launch(Product{a, 0, 0, 1}, false, s); }

hipError_t launch_grouped_linear_mxfp4(const MxLinearArgs& a, hipStream_t s) { return launch(Product{a, 0, 0, 1}, true, s); }

}  // namespace moe
