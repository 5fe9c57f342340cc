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
  int valid;     // rows that exist, 0: none
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
    // An entry that names no local expert, or rows outside the capacity, has none: whatever the list holds, nothing beyond
    // x, the weights and out is touched.
    const int t = ti / p.sub;
    r.expert = p.a.tiles[2 * t];
    r.row0 = (int64_t)p.a.tiles[2 * t + 1] + (ti - t * p.sub) * bm;
    r.valid = 0;
    if ((uint32_t)r.expert >= (uint32_t)p.a.E_loc || r.row0 < 0 || r.row0 >= p.a.R_cap) return r;
    const int64_t end = (int64_t)p.a.offsets[r.expert] + p.a.counts[r.expert];
    const int64_t left = (end < p.a.R_cap ? end : p.a.R_cap) - r.row0;
    r.valid = left < bm ? (int)(left > 0 ? left : 0) : bm;
  } else {
    r.expert = 0;
    r.row0 = (int64_t)ti * bm;
    const int64_t left = p.a.M - r.row0;
    r.valid = left < bm ? (int)left : bm;
  }
  return r;
}

// Row tiles of the list's entries.
__device__ __forceinline__ int row_tiles(const Product& p) {
  const int n = *p.a.num_tiles;
  return n > 0 ? (n < p.a.tiles_cap ? n : (int)p.a.tiles_cap) * p.sub : 0;
}

// ---------------------------------------------------------------------------
// Epilogue
// ---------------------------------------------------------------------------
// V values side by side, at any alignment their type allows (rows of odd lengths), `left` of which exist.
template <int V>
using words = uint32_t __attribute__((__vector_size__(V * 4)));

template <int V, bool F32>
__device__ __forceinline__ void load_values(const void* p, int64_t at, int left, float (&v)[V]) {
  if (left >= V) {
    if constexpr (F32) {
      typedef words<4> quad __attribute__((aligned(4)));
#pragma unroll
      for (int i = 0; i < V; i += 4) {
        const words<4> q = *reinterpret_cast<const quad*>(static_cast<const float*>(p) + at + i);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[i + e] = __builtin_bit_cast(float, (uint32_t)q[e]);
      }
    } else {
      typedef words<V / 2> halves __attribute__((aligned(2)));
      const words<V / 2> q = *reinterpret_cast<const halves*>(static_cast<const uint16_t*>(p) + at);
#pragma unroll
      for (int e = 0; e < V; ++e) v[e] = bf2f((uint16_t)(q[e >> 1] >> (16 * (e & 1))));
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      v[i] = 0.f;
      if (i < left) v[i] = F32 ? static_cast<const float*>(p)[at + i] : bf2f(static_cast<const uint16_t*>(p)[at + i]);
    }
  }
}

// through: the stores pass the caches by.  Where a wavefront writes whole lines that is faster (grouped, 49152 rows of 2048
// x 1408 in fp32 169 us instead of 187; also with the output read again at once), where rows begin inside a line slower
// (4096 x 4095 x 1024 in bf16 26 us instead of 22), and for a streamed product's 32 bytes a row too.
template <int V, bool F32>
__device__ __forceinline__ void store_values(void* p, int64_t at, int left, const float (&v)[V], bool through) {
  if (left >= V) {
    if constexpr (F32) {
      typedef words<4> quad __attribute__((aligned(4)));
#pragma unroll
      for (int i = 0; i < V; i += 4) {
        quad* to = reinterpret_cast<quad*>(static_cast<float*>(p) + at + i);
        const words<4> q = __builtin_bit_cast(words<4>, floatx4{v[i], v[i + 1], v[i + 2], v[i + 3]});
        if (through) {
          asm volatile("");  // (keeps the compiler from making one ordinary store of the two)
          __builtin_nontemporal_store(q, to);
          asm volatile("");
        } else {
          *to = q;
        }
      }
    } else {
      typedef words<V / 2> halves __attribute__((aligned(2)));
      words<V / 2> h;
#pragma unroll
      for (int e = 0; e < V / 2; ++e) h[e] = (uint32_t)f2bf_bits(v[2 * e]) | ((uint32_t)f2bf_bits(v[2 * e + 1]) << 16);
      halves* to = reinterpret_cast<halves*>(static_cast<uint16_t*>(p) + at);
      if (through) {
        asm volatile("");
        __builtin_nontemporal_store(h, to);
        asm volatile("");
      } else {
        *to = h;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < left) {
        if (F32) static_cast<float*>(p)[at + i] = v[i];
        else static_cast<uint16_t*>(p)[at + i] = f2bf_bits(v[i]);
      }
  }
}

// Activations of V columns: z (and u) are the sums, bz and bu the biases.
template <int V>
__device__ __forceinline__ void activate_row(int act, float (&z)[V], const float (&u)[V], const float (&bz)[V], const float (&bu)[V]) {
  switch (act) {
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
}

// The epilogue of C rows, V columns each from column n: sums(c, z, u) gives row c's, row(c) its index in out, or -1
// where there is none.  The rows' residuals are loaded together, ahead of the first store.
template <int V, bool F32, int C, typename Sums, typename Row>
__device__ __forceinline__ void finish(const MxLinearArgs& a, int n, bool through, Sums sums, Row row) {
  const int left = a.N - n;  // columns that exist
  if (left <= 0) return;
  float bz[V], bu[V], res[C][V];
#pragma unroll
  for (int i = 0; i < V; ++i) bz[i] = bu[i] = 0.f;
  if (a.bias) load_values<V, true>(a.bias, n, left, bz);
  if (a.bias_up) load_values<V, true>(a.bias_up, n, left, bu);
  if (a.residual)
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (row(c) >= 0) load_values<V, F32>(a.residual, row(c) * a.N + n, left, res[c]);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    if (row(c) < 0) continue;
    float z[V], u[V];
    sums(c, z, u);
    activate_row<V>(a.act, z, u, bz, bu);
    if (a.residual)
#pragma unroll
      for (int i = 0; i < V; ++i) z[i] += res[c][i];
    store_values<V, F32>(a.out, row(c) * a.N + n, left, z, through);
  }
}

// ---------------------------------------------------------------------------
// Tiles through LDS
// ---------------------------------------------------------------------------
constexpr int kXcds = 8, kCus = 256;
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
// Codes staged in registers, two LDS buffers (NS = 2): while a stage of 256 reduction indices (128 bytes a row: whole
// cache lines) is multiplied from one buffer, the next stage goes from registers into the other and the registers reload
// with the one after it.  A stage is four steps, each a matrix instruction of 64 indices per accumulator; a step's fragments are read
// during the step before, and the writes and loads are spread over the first three.  When the last step begins the
// stage has been read: there the workgroup synchronises, and the last step reads the next stage's first fragments.  The
// 128 x 128 tile takes 72 KB, so that two share a CU: 93 us at 4096 x 14336 x 2048, 131 in a ring of four stages.
//
// Bound: LDS and the matrix cores alike, and the epilogue.  A stage of the 256 x 256 tile reads 192 KB and writes 64, 2050
// cycles at 128 bytes a cycle of the 2600 to 2700 it takes, bank conflicts on top (19 % of the cycles in which LDS is active:
// the scales' reads of four bytes at a pitch of 16); its 64 matrix instructions of 32 cycles take 2048 of each SIMD.  Over a
// whole launch the matrix cores are 45 % busy, as a tile fills its CU and nothing is multiplied while its results are
// written.  Measured: 8192 x 8192 x 8192 282 us (3.9 PFLOP/s), 4096 x 14336 x 4096 SwiGLU 249 to 270 us (3.6 to 3.9).
//
// A ring of NS > 2 stages straight to LDS, for the smallest tiles, whose time is the latency of their stages: 64 x 64 takes
// 15.0 us at 128 x 4096 x 8192, 24.9 with staged codes.  Three stages, so that two or three tiles share a CU (five: 65 us
// instead of 51 for gate and up products of 64 experts, 1408 x 2048, with 48 rows each).
//
// The scales go straight to LDS for two stages at a time, 16 bytes a row: a row's bytes of one stage would each time be
// an access of their own to the row's cache line, nearly as many as the codes need (340 us instead of 294 at
// 4096 x 14336 x 4096 SwiGLU with 128-wide stages).  Lane half h takes the stage's blocks 4 h .. 4 h + 3, one for each
// step, whose scales are the bytes of the word that it reads.
template <int BM, int BN, int NMAT, int WM, int WN, int NS>
struct Tile {
  static constexpr bool RING = NS > 2;  // straight to LDS, several stages ahead
  static constexpr int NW = WM * WN;
  static constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128;
  static constexpr int STAGE = A_BYTES + NMAT * B_BYTES;
  static constexpr int ROWS = BM + NMAT * BN;  // of x, then of the matrices
  static constexpr int SCALES = NS * STAGE;    // PLACES of 16 bytes a row
  static constexpr int PLACES = RING ? NS / 2 + 1 : 2;  // (pairs of the stages from kt + 1 to kt + NS)
  static constexpr int SMEM = SCALES + PLACES * ROWS * 16;
  static constexpr int PITCH = NMAT * BN / WN + 4, EPI = 32 * PITCH * 4;  // floats a staged row, bytes of 32 of them
  static constexpr int WT_M = BM / WM, WT_N = BN / WN;
  static constexpr int TM = WT_M / 32, TN = WT_N / 32, NB = NMAT * TN;
  static constexpr int A_PIECES = BM / (8 * NW), B_PIECES = BN / (8 * NW);
  static constexpr int S_ALL = ROWS / 64, S_PIECES = (S_ALL + NW - 1) / NW;
  static constexpr int LOADS = A_PIECES + NMAT * B_PIECES;
  static_assert(BM % (8 * NW) == 0 && BN % (8 * NW) == 0 && BM % 64 == 0 && BN % 64 == 0, "whole pieces");
  static_assert(TM >= 1 && TN >= 1 && (NS - 2) * LOADS < 64, "tile");
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
    // Stage kt's codes, piece by piece: to registers and from there to LDS, or straight to LDS.  (Stages past the last
    // load from past the resources.)
    auto source = [&](int q, int kt) -> uint32_t {
      const uint32_t none = kt < nk ? (odd && kt == nk - 1 ? cut : 0) : kOut, at = (uint32_t)kt * 128;
      return ((q < A_PIECES ? off_a[q < A_PIECES ? q : 0] : off_b + (q - A_PIECES) % B_PIECES * 8 * NW * kb) + at) | none;
    };
    auto resource = [&](int q) { return q < A_PIECES ? rx : rwq[(q - A_PIECES) / B_PIECES]; };
    auto place = [&](int q, int kt) {
      const int line = q < A_PIECES ? q * NW : BM / 8 + (q - A_PIECES) / B_PIECES * (BN / 8) + (q - A_PIECES) % B_PIECES * NW;
      return smem + (kt % NS) * STAGE + (line + wave) * 1024;
    };
    u32x4 stg[RING ? 1 : LOADS];
    auto load = [&](int q, int kt) { stg[q] = __builtin_amdgcn_raw_buffer_load_b128(resource(q), source(q, kt), 0, 0); };
    auto write = [&](int q, int kt) { *reinterpret_cast<u32x4*>(place(q, kt) + lane * 16) = stg[q]; };
    // The scales of stages kt and kt + 1 (16 bytes may run into the next row's, which no stage uses).
    auto issue_scales = [&](int kt) {
#pragma unroll
      for (int q = 0; q < S_PIECES; ++q)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            rs[q], (lds_void*)(smem + SCALES + (kt / 2 % PLACES) * (ROWS * 16) + ((q * NW + wave) % S_ALL) * 1024), 16, off_s[q] + kt * 8, 0, 0, 0);
    };
    // A whole stage straight to LDS, its scales ahead of it.
    auto issue = [&](int kt) {
      if (kt % 2 == 0 && kt < nk) issue_scales(kt);
#pragma unroll
      for (int q = 0; q < LOADS; ++q)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(resource(q), (lds_void*)place(q, kt), 16, source(q, kt), 0, 0, 0);
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
      const char* st = smem + (kt % NS) * STAGE;
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
      const char* sc = smem + SCALES + (kt / 2 % PLACES) * (ROWS * 16) + (kt % 2) * 8 + half * 4;
#pragma unroll
      for (int i = 0; i < TM; ++i) f.a[i] = *reinterpret_cast<const int*>(sc + (wm * WT_M + i * 32 + l32) * 16);
#pragma unroll
      for (int j = 0; j < NB; ++j)
        f.b[j] = *reinterpret_cast<const int*>(sc + (BM + (j / TN) * BN + wn * WT_N + (j % TN) * 32 + l32) * 16);
    };
    auto blank = [&](Scales& s, int kt) {  // (no scales past the row's end; the codes are zeros)
      if (odd && kt == nk - 1 && half) {
#pragma unroll
        for (int i = 0; i < TM; ++i) s.a[i] = 0;
#pragma unroll
        for (int j = 0; j < NB; ++j) s.b[j] = 0;
      }
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
      if constexpr (!RING)
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
    if constexpr (RING) {
#pragma unroll
      for (int kt = 0; kt < NS; ++kt) issue(kt);
      wait_vmcnt<(NS - 1) * LOADS>();
      ring_barrier();
      struct Whole {
        Frags f[4];
        Scales s;
      };
      Whole w[2];
      auto read_stage = [&](Whole& v, int kt) {
#pragma unroll
        for (int q = 0; q < 4; ++q) read(v.f[q], kt, q);
        read_scales(v.s, kt);
      };
      auto stage = [&](Whole& cur, Whole& next, int kt) {
        wait_lgkm0();                     // this wavefront's reads of stage kt are done
        wait_vmcnt<(NS - 2) * LOADS>();   // its loads of stage kt + 1, with their scales, have landed
        ring_barrier();                   // so are and have all others'
        issue(kt + NS);                   // into the place of stage kt
        read_stage(next, kt + 1);
        blank(cur.s, kt);
        multiply(integral_constant<int, 0>{}, cur.f[0], cur.s);
        multiply(integral_constant<int, 1>{}, cur.f[1], cur.s);
        multiply(integral_constant<int, 2>{}, cur.f[2], cur.s);
        multiply(integral_constant<int, 3>{}, cur.f[3], cur.s);
      };
      read_stage(w[0], 0);
      for (int kt = 0; kt < nk; kt += 2) {
        stage(w[0], w[1], kt);
        if (kt + 1 < nk) stage(w[1], w[0], kt + 1);
      }
      wait_vmcnt<0>();  // (the empty stages' writes to LDS)
      wait_lgkm0();
    } else {
      Frags f[2];
      Scales sc, next;
      issue_scales(0);
      __builtin_amdgcn_sched_barrier(0);
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
        blank(sc, kt);
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
      if (a.out_f32) store_rows<4, true>(a, rw, sm, r0, n0 + wn * WT_N, lane);
      else store_rows<8, false>(a, rw, sm, r0, n0 + wn * WT_N, lane);
    }
  }

  // The epilogue of 32 staged rows from row r0 of the tile: V columns a lane, up to eight rows of a lane together (one by
  // one, 4096 x 14336 x 512 with an fp32 residual took 217 us instead of 130).
  template <int V, bool F32>
  static __device__ __forceinline__ void store_rows(const MxLinearArgs& a, const Rows& rw, const float* sm, int r0, int n0,
                                                    int lane) {
    constexpr int LPR = WT_N / V, STEP = 64 / LPR, C = 32 / STEP;  // lanes a row, rows at a time
    const int c0 = lane % LPR * V, r = lane / LPR;
    finish<V, F32, C>(
        a, n0 + c0, a.N % (F32 ? 16 : 32) == 0,
        [&](int c, float (&z)[V], float (&u)[V]) {
          const float* s = sm + (r + c * STEP) * PITCH + c0;
#pragma unroll
          for (int v = 0; v < V; v += 4) {
            const floatx4 p = *reinterpret_cast<const floatx4*>(s + v);
            const floatx4 q = NMAT == 2 ? *reinterpret_cast<const floatx4*>(s + WT_N + v) : p;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              z[v + e] = p[e];
              u[v + e] = q[e];
            }
          }
        },
        [&](int c) -> int64_t {
          const int q = r0 + r + c * STEP;
          return q < rw.valid ? rw.row0 + q : -1;
        });
  }
};

template <int BM, int BN, int NMAT, int WM, int WN, int NS, bool GROUPED>
__global__ __launch_bounds__(WM* WN * 64) void tile_kernel(Product p) {
  using T = Tile<BM, BN / NMAT, NMAT, WM, WN, NS>;
  __shared__ __attribute__((aligned(1024))) char smem[T::SMEM];
  const int mt = GROUPED ? row_tiles(p) : p.mt;
  if ((int)blockIdx.x >= mt * p.nt) return;
  int ti, tj;
  tile_of(blockIdx.x, mt, p.nt, ti, tj);
  const Rows rw = rows_of<GROUPED>(p, ti, BM);
  if (rw.valid == 0) return;
  T::template run<GROUPED>(smem, p, rw, tj * (BN / NMAT));
}

// ---------------------------------------------------------------------------
// Few rows: the weights stream from global memory into the matrix instructions' registers
// ---------------------------------------------------------------------------
// Up to 16 MB rows by 16 columns a workgroup; its wavefronts take turns at units of 512 reduction indices and add up
// through LDS.  v_mfma_scale_f32_16x16x128: lane l holds block l / 16 of four of row l % 16, so a load of 16 bytes a
// lane is 64 contiguous bytes of each of 16 rows, and a unit's 16 scale bytes of a row come as one load.
//
// With at most four rows one load has x for the four steps of a unit, step s in columns 4 s .. 4 s + 3, and a step's
// fragment is that register shifted by DPP (a column's result depends on its own row alone: the other columns hold
// anything); a load a step would cost as many accesses as the weights.
//
// Bound: HBM where there are weights enough (64 experts' 1408 x 2048 gate and up products, six rows each, 38 us, 5.1 TB/s),
// else the units' latency (one row of 2048 x 7168 SwiGLU 7.0 us).
constexpr int kStreamWaves = 4;

template <int MB, int NMAT, bool GROUPED, bool FOUR>
__device__ __forceinline__ void stream_rows(const Product& p, const Rows& rw, int n0, float* red) {
  constexpr int RED = NMAT * MB * 256;  // floats of a wavefront's sums
  constexpr int XL = FOUR ? 1 : 4, NWV = kStreamWaves;
  const MxLinearArgs& a = p.a;
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
    const int r = FOUR ? l16 & 3 : i * 16 + l16;
    uint32_t row = (uint32_t)r;
    bool in = r < rw.valid;
    if (gather) {
      const int src = in ? a.row_src[rw.row0 + r] : -1;
      row = (uint32_t)src / (uint32_t)a.topk;
      in = src >= 0 && row < a.M;
    }
    ox[i] = in ? row * (uint32_t)kb + g * 16 + (FOUR ? (l16 >> 2) * 64 : 0) : kOut;
    oxs[i] = in ? row * (uint32_t)sb : kOut;
  }
  const uint32_t ow = (uint32_t)(l16 * kb + g * 16), ows = (uint32_t)(l16 * sb);

  floatx4 acc[NMAT][MB];
#pragma unroll
  for (int m = 0; m < NMAT; ++m)
#pragma unroll
    for (int i = 0; i < MB; ++i) acc[m][i] = floatx4{0.f, 0.f, 0.f, 0.f};

  struct Unit {
    u32x4 w[NMAT][4], ws[NMAT], x[MB][XL], xs[MB];
  };
  // (steps past the row's end load from past the resource; the scales of a unit may run into the next row's, which no
  // step uses; loads marked as streaming, which leave no half lines for the next step, took 409 us there)
  auto load = [&](Unit& v, int u) {
    const int steps = (a.K - u * 512) / 128;  // (4 but for the last unit; none past it)
#pragma unroll
    for (int m = 0; m < NMAT; ++m) {
#pragma unroll
      for (int s = 0; s < 4; ++s)
        v.w[m][s] = __builtin_amdgcn_raw_buffer_load_b128(rwq[m], s < steps ? ow + u * 256 + s * 64 : kOut, 0, 0);
      v.ws[m] = __builtin_amdgcn_raw_buffer_load_b128(rws[m], steps > 0 ? ows + u * 16 : kOut, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < MB; ++i) {
#pragma unroll
      for (int s = 0; s < XL; ++s)
        v.x[i][s] = __builtin_amdgcn_raw_buffer_load_b128(rx, (FOUR ? l16 >> 2 : s) < steps ? ox[i] + u * 256 + s * 64 : kOut, 0, 0);
      v.xs[i] = __builtin_amdgcn_raw_buffer_load_b128(rxs, steps > 0 ? oxs[i] + u * 16 : kOut, 0, 0);
    }
  };
  auto multiply = [&](const Unit& v, int u) {
    const int steps = (a.K - u * 512) / 128;
    auto step = [&](auto s_) {
      constexpr int S = decltype(s_)::value;
      const bool in = S < steps;  // (past the row's end the codes are zeros, and so are their scales)
#pragma unroll
      for (int m = 0; m < NMAT; ++m)
#pragma unroll
        for (int i = 0; i < MB; ++i) {
          const u32x4 t = FOUR ? shifted<FOUR ? 4 * S : 0>(v.x[i][0]) : v.x[i][FOUR ? 0 : S];
          acc[m][i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
              widen(v.w[m][S]), widen(t), acc[m][i], kFp4, kFp4, 0, in ? (int)(v.ws[m][S] >> (8 * g)) : 0, 0,
              in ? (int)(v.xs[i][S] >> (8 * g)) : 0);
        }
    };
    step(std::integral_constant<int, 0>{});
    step(std::integral_constant<int, 1>{});
    step(std::integral_constant<int, 2>{});
    step(std::integral_constant<int, 3>{});
  };
  // One unit's registers, loaded again as soon as they are multiplied: a second unit's took 340 us where this takes 260
  // for gate and up products of 64 experts of 2048 x 7168, 16 rows each, because fewer wavefronts fit.  (The loads stand
  // at the loop's end so that they are all issued together.)
  Unit q;
  load(q, wave);
  for (int u = wave; u < units; u += NWV) {
    multiply(q, u);
    if (u + NWV < units) load(q, u + NWV);
  }
#pragma unroll
  for (int m = 0; m < NMAT; ++m)
#pragma unroll
    for (int i = 0; i < MB; ++i) *reinterpret_cast<floatx4*>(red + wave * RED + (m * MB + i) * 256 + lane * 4) = acc[m][i];
  __syncthreads();
  // Lane l of a partial sum: row l % 16, columns 4 (l / 16) + 0..3.  One wavefront per 16 rows, in the units' order.
  if (wave < MB) {
    floatx4 z = {0.f, 0.f, 0.f, 0.f}, v = z;
#pragma unroll
    for (int w = 0; w < NWV; ++w) {
      const float* s = red + w * RED + wave * 256 + lane * 4;
      z += *reinterpret_cast<const floatx4*>(s);
      if (NMAT == 2) v += *reinterpret_cast<const floatx4*>(s + MB * 256);
    }
    const int r = wave * 16 + l16;
    auto sums = [&](int, float (&zv)[4], float (&uv)[4]) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        zv[i] = z[i];
        uv[i] = v[i];
      }
    };
    auto row = [&](int) -> int64_t { return r < rw.valid ? rw.row0 + r : -1; };
    if (a.out_f32) finish<4, true, 1>(a, n0 + g * 4, false, sums, row);
    else finish<4, false, 1>(a, n0 + g * 4, false, sums, row);
  }
}

template <int MB, int NMAT, bool GROUPED>
__global__ __launch_bounds__(kStreamWaves * 64) void stream_kernel(Product p) {
  __shared__ float red[kStreamWaves * NMAT * MB * 256];
  const int ti = blockIdx.x / p.nt, n0 = (int)(blockIdx.x % p.nt) * 16;
  if (GROUPED && ti >= row_tiles(p)) return;
  const Rows rw = rows_of<GROUPED>(p, ti, 16 * MB);
  if (rw.valid == 0) return;
  if (MB == 1 && rw.valid <= 4) stream_rows<MB, NMAT, GROUPED, MB == 1>(p, rw, n0, red);
  else stream_rows<MB, NMAT, GROUPED, false>(p, rw, n0, red);
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
#define MOE_TILE(BM_, BN_, BN2_, WM_, WN_, NS_)                                                            \
  do {                                                                                                     \
    if (grouped && dual) MOE_LAUNCH((tile_kernel<BM_, BN2_, 2, WM_, WN_, NS_, true>), WM_* WN_ * 64);      \
    if (grouped) MOE_LAUNCH((tile_kernel<BM_, BN_, 1, WM_, WN_, NS_, true>), WM_* WN_ * 64);               \
    if (dual) MOE_LAUNCH((tile_kernel<BM_, BN2_, 2, WM_, WN_, NS_, false>), WM_* WN_ * 64);                \
    MOE_LAUNCH((tile_kernel<BM_, BN_, 1, WM_, WN_, NS_, false>), WM_* WN_ * 64);                           \
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
  const int nk = (p.a.K + kStage - 1) / kStage;
  // Tiles: the kind that takes least, in us as fitted to 77 products of 64 to 49152 rows, 512 to 14336 indices, bf16 and
  // fp32 outputs (its choice is 0.4 % above the best kind on average, 6 % at most, over 71 of them).  A CU holds one of the two large kinds
  // at a time, which run in whole rounds.  It holds two or three of the small ones: rounds run into each other, and their
  // stages overlap but for the latency of a tile alone.
  struct Kind {
    int bm, bn;
    bool whole;
    float stage, tile, alone, out16, out32, fixed;  // us a stage, a tile, a stage of one tile alone, a MB of out, a launch
  };
  const Kind kinds[] = {{256, 256, true, 1.37f, 7.8f, 0.f, 0.15f, 0.18f, 1.8f},
                        {256, 128, true, 0.94f, 4.1f, 0.f, 0.16f, 0.19f, 2.4f},
                        {128, 128, false, 0.68f, 0.5f, 0.62f, 0.095f, 0.15f, 5.6f},
                        {64, dual ? 128 : 64, false, dual ? 0.42f : 0.23f, 0.f, dual ? 0.5f : 0.3f, 0.34f, 0.24f, 4.6f}};
  const float out_rows = (float)(grouped ? p.a.tiles_cap * rows : rows);
  const float out_mb = out_rows * p.a.N * (p.a.out_f32 ? 4e-6f : 2e-6f) * (p.a.residual ? 2 : 1);
  int best = 3;
  float least = 0.f;
  for (int i = 3; i >= 0; --i) {
    const Kind& k = kinds[i];
    if (k.bm > rows && i < 3) continue;
    tiles(k.bm, k.bn / mats);
    const int64_t n = (int64_t)p.mt * p.nt;
    const float x = (float)n / kCus, up = (float)((n + kCus - 1) / kCus), rounds = k.whole ? up : 0.5f * (x + up);
    const float work = rounds * (nk * k.stage + k.tile), alone = nk * k.alone;
    const float t = (work > alone ? work : alone) + out_mb * (p.a.out_f32 ? k.out32 : k.out16) + k.fixed;
    // Grouped, a capacity of at least a round takes the largest square tiles that fit tile_m (64 experts with 192 rows each,
    // 2048 x 1408, fp32, tile_m 256: 70 us, 86 in tiles of 128; the capacity says little about the tiles that have rows).
    if (i == 3 || t < least || (grouped && i != 1 && x >= 1.f)) {
      best = i;
      least = t;
    }
  }
  // Few rows: streamed where that takes less, us by the megabyte of codes as measured on 29 MB (17 rows of 4096 x 14336
  // 11.7 us, 21.5 in tiles; of 14336 x 4096 13.3, 10.2 in tiles).  Over 30 products of 17 to 64 rows the choice is 3 % above
  // the best on average, 23 % at most (33 rows of 4096 x 14336: 21.7 in tiles, 17.7 streamed).  Grouped, tiles are never cut below 64 rows.
  const float mb_codes = (float)p.a.N * p.a.K * mats * 0.5e-6f;
  if (rows <= 16 || (grouped && rows < 64) || (!grouped && rows <= 32 && 5.f + 0.38f * mb_codes < least) ||
      (!grouped && rows <= 64 && 6.f + 0.65f * mb_codes < least)) {
    const int mb = rows <= 16 ? 1 : rows <= 32 ? 2 : 4;
    tiles(16 * mb, 16);
    if (mb == 1) MOE_STREAM(1);
    if (mb == 2) MOE_STREAM(2);
    if (dual) MOE_LAUNCH((stream_kernel<4, 2, false>), kStreamWaves * 64);
    MOE_LAUNCH((stream_kernel<4, 1, false>), kStreamWaves * 64);
  }
  tiles(kinds[best].bm, kinds[best].bn / mats);
  // (2 x 4 wavefronts have half as long runs of a row to store: 113 us instead of 96 at 4096 x 14336 x 2048)
  if (best == 0) MOE_TILE(256, 256, 256, 4, 2, 2);
  if (best == 1) MOE_TILE(256, 128, 128, 4, 2, 2);
  if (best == 2) MOE_TILE(128, 128, 128, 4, 2, 2);
  MOE_TILE(64, 64, 128, 2, 2, 3);
#undef MOE_LAUNCH
#undef MOE_TILE
#undef MOE_STREAM
}

}  // namespace

hipError_t launch_linear_mxfp4(const MxLinearArgs& a, hipStream_t s) { return launch(Product{a, 0, 0, 1}, false, s); }

hipError_t launch_grouped_linear_mxfp4(const MxLinearArgs& a, hipStream_t s) { return launch(Product{a, 0, 0, 1}, true, s); }

}  // namespace moe
