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
// V values of one row from column n: bias, activation, residual, rounding, stores.  `at` is the element's index in out.
template <int V>
__device__ __forceinline__ void finish(const MxLinearArgs& a, int64_t at, int n, float (&z)[V], const float (&u)[V]) {
  constexpr int W = V < 8 ? V : 8;  // bf16 values per access
  const int left = a.N - n;         // columns that exist
  if (left <= 0) return;
  const bool whole = left >= V && a.N % 8 == 0;  // (then every row's groups of V are 16-byte aligned)
  float bz[V], bu[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    bz[i] = a.bias && i < left ? a.bias[n + i] : 0.f;
    bu[i] = a.bias_up && i < left ? a.bias_up[n + i] : 0.f;
  }
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
// together are lanes 0-3, 12-15, 20-27 or 4-11, 16-19, 28-31 (and 32 on): this spreads both the token fragment's rows
// (lane) and the weight fragment's (weight_row) over all 64 banks.
__device__ __forceinline__ constexpr int swz(int row) { return (row >> 1) & 7; }

// The weight row, of a block of 32, that feeds row r of the matrix instruction.  Result element i of lane half h is
// instruction row 8 (i / 4) + 4 h + i % 4; fed by weight row 16 h + i, a lane's 16 results are 16 columns side by side.
__device__ __forceinline__ constexpr int weight_row(int r) { return 16 * ((r >> 2) & 1) + 4 * (r >> 3) + (r & 3); }

// BM rows by BN columns (NMAT = 2: BN of each matrix), WM x WN wavefronts.
//
// A stage of 256 reduction indices (128 bytes a row, and 8 scale bytes) goes straight from global memory to one of two
// LDS buffers while the other is multiplied.  Lane half h takes the stage's blocks 4 h .. 4 h + 3, one for each of four
// instructions, so that the four scales are the bytes of one word, selected by the instruction.
template <int BM, int BN, int NMAT, int WM, int WN>
struct Tile {
  static constexpr int NW = WM * WN;
  static constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128;
  static constexpr int SA = A_BYTES + NMAT * B_BYTES, SB = SA + BM * 8;  // the scales' places in a stage
  static constexpr int STAGE = SB + NMAT * BN * 8;
  static constexpr int WT_M = BM / WM, WT_N = BN / WN;
  static constexpr int TM = WT_M / 32, TN = WT_N / 32, NB = NMAT * TN;
  static constexpr int A_PIECES = BM / (8 * NW), B_PIECES = BN / (8 * NW);
  static_assert(BM == 32 * NW && NMAT * BN == 32 * NW, "a wavefront loads 32 rows' scales of either operand");
  static_assert(A_PIECES >= 1 && B_PIECES >= 1 && TM >= 1 && TN >= 1, "tile too small for the wavefronts");

  template <bool GROUPED>
  static __device__ __forceinline__ void run(char* smem, const Product& p, const Rows& rw, int n0) {
    const MxLinearArgs& a = p.a;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN, l32 = lane & 31, half = lane >> 5;
    const int kb = a.K / 2, sb = a.K / 32, nk = (a.K + kStage - 1) / kStage;
    const bool gather = GROUPED && a.row_src != nullptr;
    const int cols = a.N - n0 < BN ? a.N - n0 : BN;

    // Resources: x's rows (gathered: all of x), the tile's weight rows.
    const int64_t x0 = gather ? 0 : rw.row0, xr = gather ? a.M : rw.valid;
    const __amdgpu_buffer_rsrc_t rx = make_rsrc(a.x.q + x0 * kb, xr * kb), rxs = make_rsrc(a.x.s + x0 * sb, xr * sb);
    const int64_t w0 = (int64_t)rw.expert * a.N + n0;
    const __amdgpu_buffer_rsrc_t rwq[2] = {make_rsrc(a.w.q + w0 * kb, (int64_t)cols * kb),
                                           make_rsrc((NMAT == 2 ? a.w_up.q : a.w.q) + w0 * kb, (int64_t)cols * kb)};
    // This lane's offsets.  Codes: rows of 8 lanes, 16 bytes each.  Scales: rows of 2 lanes, a word each; the wavefront
    // loads those of 32 rows of x and of 32 rows of the matrices one after the other.
    const int r_in = lane >> 3, chunk = (lane & 7) ^ swz(wave * 8 + r_in);
    uint32_t off_a[A_PIECES], off_b = (uint32_t)((wave * 8 + r_in) * kb + chunk * 16);
    uint32_t off_sa, off_sb;
#pragma unroll
    for (int q = 0; q < A_PIECES; ++q) {
      const int r = (q * NW + wave) * 8 + r_in;
      uint32_t row = (uint32_t)r;
      bool in = r < rw.valid;
      if (gather) {
        const int src = in ? a.row_src[rw.row0 + r] : -1;
        row = (uint32_t)src / (uint32_t)a.topk;
        in = src >= 0 && row < a.M;
      }
      off_a[q] = in ? row * (uint32_t)kb + chunk * 16 : kOut;
    }
    {
      const int r = wave * 32 + (lane >> 1);
      uint32_t row = (uint32_t)r;
      bool in = r < rw.valid;
      if (gather) {
        const int src = in ? a.row_src[rw.row0 + r] : -1;
        row = (uint32_t)src / (uint32_t)a.topk;
        in = src >= 0 && row < a.M;
      }
      off_sa = in ? row * (uint32_t)sb + (lane & 1) * 4 : kOut;
      off_sb = (uint32_t)((r % BN) * sb + (lane & 1) * 4);
    }
    const bool up_scales = NMAT == 2 && wave * 32 >= BN;
    const __amdgpu_buffer_rsrc_t rws = make_rsrc((up_scales ? a.w_up.s : a.w.s) + w0 * sb, (int64_t)cols * sb);
    // K is a multiple of 128: where the last stage is half a stage, the later half of each row reads zeros.
    const bool odd = (a.K & 128) != 0;
    const uint32_t cut_c = chunk >= 4 ? kOut : 0, cut_s = (lane & 1) ? kOut : 0;

    auto issue = [&](int kt, int buf) {
      char* st = smem + buf * STAGE;
      const bool cut = odd && kt == nk - 1;
      const uint32_t at = (uint32_t)kt * 128, cc = cut ? cut_c : 0, cs = cut ? cut_s : 0;
#pragma unroll
      for (int q = 0; q < A_PIECES; ++q)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (lds_void*)(st + (q * NW + wave) * 1024), 16, (off_a[q] + at) | cc, 0, 0, 0);
#pragma unroll
      for (int m = 0; m < NMAT; ++m)
#pragma unroll
        for (int q = 0; q < B_PIECES; ++q)
          __builtin_amdgcn_raw_ptr_buffer_load_lds(rwq[m], (lds_void*)(st + A_BYTES + m * B_BYTES + (q * NW + wave) * 1024), 16,
                                                   (off_b + q * 8 * NW * kb + at) | cc, 0, 0, 0);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rxs, (lds_void*)(st + SA + wave * 256), 4, (off_sa + kt * 8) | cs, 0, 0, 0);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rws, (lds_void*)(st + SB + wave * 256), 4, (off_sb + kt * 8) | cs, 0, 0, 0);
    };

    floatx16 acc[NB][TM];
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[j][i][v] = 0.f;
    const int brow = weight_row(l32);

    issue(0, 0);
    wait_vmcnt<0>();
    ring_barrier();
    for (int kt = 0; kt < nk; ++kt) {
      const char* st = smem + (kt & 1) * STAGE;
      if (kt + 1 < nk) issue(kt + 1, (kt & 1) ^ 1);
      int sa[TM], sw[NB];
#pragma unroll
      for (int i = 0; i < TM; ++i) sa[i] = *reinterpret_cast<const int*>(st + SA + (wm * WT_M + i * 32 + l32) * 8 + half * 4);
#pragma unroll
      for (int j = 0; j < NB; ++j)
        sw[j] = *reinterpret_cast<const int*>(st + SB + ((j / TN) * BN + wn * WT_N + (j % TN) * 32 + brow) * 8 + half * 4);
#define MOE_STEP(S_)                                                                                              \
  {                                                                                                               \
    u32x4 fa[TM], fb[NB];                                                                                         \
    _Pragma("unroll") for (int j = 0; j < NB; ++j) {                                                              \
      const int row = wn * WT_N + (j % TN) * 32 + brow;                                                           \
      fb[j] = *reinterpret_cast<const u32x4*>(st + A_BYTES + (j / TN) * B_BYTES + row * 128 + (((half * 4 + S_) ^ swz(row)) << 4)); \
    }                                                                                                             \
    _Pragma("unroll") for (int i = 0; i < TM; ++i) {                                                              \
      const int row = wm * WT_M + i * 32 + l32;                                                                   \
      fa[i] = *reinterpret_cast<const u32x4*>(st + row * 128 + (((half * 4 + S_) ^ swz(row)) << 4));              \
    }                                                                                                             \
    _Pragma("unroll") for (int j = 0; j < NB; ++j) _Pragma("unroll") for (int i = 0; i < TM; ++i)                 \
        acc[j][i] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(widen(fb[j]), widen(fa[i]), acc[j][i], kFp4, kFp4, S_, \
                                                                    sw[j], S_, sa[i]);                            \
  }
      MOE_STEP(0)
      MOE_STEP(1)
      MOE_STEP(2)
      MOE_STEP(3)
#undef MOE_STEP
      wait_vmcnt<0>();
      wait_lgkm0();
      ring_barrier();
    }

    // Lane: row l32 of each 32-row block, 16 columns side by side of each 32-column block.  One block at a time in a
    // loop, so that the activations' code is there once.
    constexpr int BLOCKS = TN * TM;
#pragma unroll 1
    for (int b = 0; b < BLOCKS; ++b) {
      floatx16 z = acc[0][0], u = acc[0][0];
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int i = 0; i < TM; ++i)
          if (j * TM + i == b) {
            z = acc[j][i];
            if (NMAT == 2) u = acc[NB - TN + j][i];
          }
      const int r = wm * WT_M + (b % TM) * 32 + l32;
      if (r >= rw.valid) continue;
      const int n = n0 + wn * WT_N + (b / TM) * 32 + half * 16;
      float zv[16], uv[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        zv[i] = z[i];
        uv[i] = u[i];
      }
      finish<16>(a, (rw.row0 + r) * a.N + n, n, zv, uv);
    }
  }
};

template <int BM, int BN, int NMAT, int WM, int WN, bool GROUPED>
__global__ __launch_bounds__(WM* WN * 64) void tile_kernel(Product p) {
  using T = Tile<BM, BN / NMAT, NMAT, WM, WN>;
  __shared__ __attribute__((aligned(1024))) char smem[2 * T::STAGE];
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
