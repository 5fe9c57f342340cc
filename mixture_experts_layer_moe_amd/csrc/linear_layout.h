// How the dense projection divides its products into tiles and launches, and where the tiles' loads lie: arithmetic
// alone, so that a host test can ask for a size's tiles and walk every lane of every stage.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace moe {

constexpr int BK = 64;                  // reduction indices per stage
constexpr uint32_t kOut = 0x80000000u;  // a byte offset past every resource

// Rows operand: LDS row of 128 B per operand row, 16-byte chunk index XORed with row / 2.  A fragment read takes 16
// rows at four chunks; the 16 lanes served together are rows 0-3 and 12-15 at one chunk and rows 4-11 at the next
// one (or the other way round), which this spreads over all 64 banks, as it does 16 rows at one chunk.
constexpr int swz(int row) { return (row >> 1) & 7; }
// Paired rows operand (the forward product's weights): a fragment's rows are 8 (lane / 4 % 4) + lane % 4 of a block of
// 32, plus 4 for its partner, so that a lane's results of both are eight columns side by side: outputs are written 16
// bytes at a time.  The 16 lanes served together are again at two neighbouring chunks.
constexpr int swz_p(int row) { return ((row >> 1) & 1) | ((row >> 3) & 3) << 1; }
// Columns operand of C columns: LDS row of 2 C bytes per reduction index; half a wavefront of a transposing read
// takes 32 bytes of each of the rows r..r + 3 and r + 8..r + 11, so the 64-byte unit is XORed with the row and the
// 32-byte half of it with row / 8 to spread those over all 64 banks.
template <int C>
constexpr int swz_t(int r) {
  return (C >= 128 ? (r & 3) << 2 : ((r >> 1) & 1) << 2) | ((r >> 3) & 1) << 1;
}

// A lane's loads of C rows (COLS: columns) of an operand from c0 on, staged by NW wavefronts; the operand has `extent`
// rows (columns) and R reduction indices per segment, ld elements between stored rows.  Stage kt is read through a
// resource of bytes(kt) bytes at its first element, piece p of this lane at offset(kt) + p step.  Rows and reduction
// indices past the operand's end lie outside of the resource.
template <bool COLS, int C, int NW, bool PAIRED>
struct SourceMap {
  int64_t adv;         // bytes between stages
  int full, tail;      // resource bytes of a stage, and of a segment's last stage
  int seg, k1;         // stages per segment; stages from k1 on are empty
  uint32_t off, step;  // this lane's byte offset of piece 0, and between pieces
  int klim;            // rows operand: stages whose chunk of this lane lies before the reduction's end

  constexpr SourceMap(int64_t ld, int64_t extent, int64_t R, int64_t c0, int seg_, int k1_, int wave, int lane)
      : adv(0), full(0), tail(0), seg(seg_), k1(k1_), off(0), step(0), klim(0) {
    if (!COLS) {
      adv = BK * 2;
      const int left = (int)(extent - c0 < C ? extent - c0 : C);
      const int width = R < BK ? (int)R : BK;  // (BK columns of the last row would hold row `left` where R = ld < BK)
      full = tail = (int)(((left - 1) * ld + width) * 2);
      const int row = wave * 8 + (lane >> 3), chunk = (lane & 7) ^ (PAIRED ? swz_p(row) : swz(row));
      off = (uint32_t)((row * ld + chunk * 8) * 2);
      step = (uint32_t)(8 * NW * ld * 2);  // (8 NW rows on, the swizzle is the same)
      klim = (int)((R - chunk * 8 + BK - 1) / BK);
    } else {
      constexpr int LPR = C / 8;  // lanes per LDS row
      adv = BK * ld * 2;
      const int last = (int)(R - (int64_t)(seg - 1) * BK);  // reduction indices in a segment's last stage
      full = (int)(((BK - 1) * ld + (extent - c0)) * 2);
      tail = (int)(((last - 1) * ld + (extent - c0)) * 2);
      const int r = wave * (64 / LPR) + lane / LPR, chunk = (lane % LPR) ^ swz_t<C>(r);
      off = c0 + chunk * 8 < extent ? (uint32_t)((r * ld + chunk * 8) * 2) : kOut;
      step = (uint32_t)(NW * (64 / LPR) * ld * 2);
    }
  }
  constexpr int bytes(int kt) const {
    const bool short_stage = COLS && (kt == seg - 1 || kt == 2 * seg - 1);
    return kt >= k1 ? 0 : short_stage ? tail : full;
  }
  constexpr uint32_t offset(int kt) const { return COLS || kt < klim ? off : kOut; }
};

// ---------------------------------------------------------------------------
// Tiles and slices
// ---------------------------------------------------------------------------
// Tile kinds: rows, columns staged per stage (of one matrix, or half of each of two), wavefronts, workgroups per CU.
// A stage reads (BM + BN) x 128 bytes for BM BN x 64 products, so large tiles run at a higher rate (the us per stage in
// make_plan: 1.43, 1.15, 1.01 and 0.84 PFLOP/s) and small ones fill the chip when there are few: 1024 x 2048 x 512
// takes 8.5 us with 64-row tiles, 4096 x 2048 x 2816 49 us with 256x128 (one round of 256) where 256x256 tiles keep
// half of the CUs idle.
struct Kind {
  int bm, bn, wm, wn, per_cu;
  constexpr int threads() const { return wm * wn * 64; }
};
constexpr Kind kKinds[] = {{256, 256, 2, 4, 1}, {256, 128, 4, 2, 1}, {128, 128, 2, 2, 2}, {64, 128, 2, 2, 3}};
constexpr int kNumKinds = 4;

inline int stages(int64_t R) { return (int)((R + BK - 1) / BK); }

// How a launch runs: its tile kind and, per product, the slices of the reduction.
struct Size {
  int64_t M;
  int N, nk;
};
struct Plan {
  int kind;
  int S[3];
  int64_t tiles[3];
  size_t part_bytes[3];  // fp32 sums of a split product
  double time;           // estimated us
};

constexpr int kMaxSlices = 16;

// Picks the tile kind and slices with the least estimated time, from measured figures of each kind (products of one
// to seven rounds, K 64 to 4096): a CU runs its share of the launch's workgroups, per_cu of them at a time, a stage of r
// workgroups taking max(latency, r * rate), plus a fixed cost per workgroup; a split adds the second launch and its
// traffic.  For a single product the rate is that of the CUs in use, since the others' idling raises their clock (3000 x
// 3000 x 1000: 144 tiles of 256x256 take 28 us, the 64x128 tiles chosen without this 39); in the backward pass's launch
// other products fill them.
inline Plan make_plan(const Size* z, int n, int nmat, bool split, int cus) {
  constexpr double kRate[] = {1.5, 0.93, 0.53, 0.32};      // us a stage and workgroup, CU full
  constexpr double kLatency[] = {1.1, 0.73, 0.56, 0.42};   // us a stage, at least
  constexpr double kFixed[] = {9.0, 6.0, 5.0, 3.5};        // us a workgroup: first stage's latency and epilogue
  constexpr double kSecond = 5.0, kBytes = 4.0e6;    // us of the second launch; bytes per us of its traffic
  constexpr double kUneven = 2.6;  // two workgroups a CU on average, where three fit: many CUs get three
  constexpr double kMaxThreads = 4294967295.0 - (1 << 25);  // of a grid, less the bias sums' (N <= 2^20)
  Plan best{};
  best.time = 1e30;
  for (int kind = 0; kind < kNumKinds; ++kind) {
    const int bm = kKinds[kind].bm, bn = kKinds[kind].bn / nmat, occ = kKinds[kind].per_cu;
    for (int S = 1; S <= (split ? kMaxSlices : 1); ++S) {
      Plan p{};
      p.kind = kind;
      double blocks = 0, work = 0, bytes = 0;
      int longest = 0;
      bool any = false;
      for (int q = 0; q < n; ++q) {
        p.tiles[q] = ((z[q].M + bm - 1) / bm) * ((z[q].N + bn - 1) / bn);
        const int most = z[q].nk / 4 < 1 ? 1 : z[q].nk / 4;  // at least four stages a slice
        p.S[q] = S < most ? S : most;
        any |= p.S[q] == S;
        const int per = (z[q].nk + p.S[q] - 1) / p.S[q];
        blocks += (double)p.tiles[q] * p.S[q];
        work += (double)p.tiles[q] * p.S[q] * per;
        longest = per > longest ? per : longest;
        if (p.S[q] > 1) {
          p.part_bytes[q] = (size_t)p.tiles[q] * p.S[q] * bm * nmat * bn * 4;
          bytes += 2.0 * p.part_bytes[q];
        }
      }
      if (!any || blocks * kKinds[kind].threads() > kMaxThreads) continue;
      const double per_block = work / blocks;          // stages of an average workgroup
      int64_t left = (int64_t)((blocks + cus - 1) / cus);  // workgroups of the fullest CU
      double t = 0, rest = blocks;
      while (left > 0) {
        const int r = left < occ ? (int)left : occ;
        double at_once = r;
        if (n == 1) at_once = r == 1 && rest < cus ? rest / cus : r == 2 && occ == 3 ? kUneven : r;
        const double stage = kLatency[kind] > at_once * kRate[kind] ? kLatency[kind] : at_once * kRate[kind];
        t += (t == 0 ? longest : per_block) * stage + kFixed[kind];
        left -= r;
        rest -= (double)r * cus;
      }
      if (bytes > 0) t += kSecond + bytes / kBytes;
      p.time = t;
      if (t < best.time) best = p;
    }
  }
  return best;
}

inline size_t part_bytes(const Plan& p, int n) {
  size_t b = 0;
  for (int q = 0; q < n; ++q) b += p.part_bytes[q];
  return b;
}

constexpr int kSkinnyRows = 16;  // up to here moe_linear streams the weights

// How moe_linear runs: `rest` last rows stream the weights, the rows before them (if any) go through tiles.  A few
// rows over a multiple of the tile would cost a whole row of tiles (4099 x 2048 x 2816: 66 us against 50 + 7).
struct ForwardPlan {
  int rest;
  Plan tiles;
};
inline ForwardPlan forward_plan(int64_t M, int N, int K, int nmat, bool split, int cus) {
  ForwardPlan f{};
  if (M <= kSkinnyRows) {
    f.rest = (int)M;
    return f;
  }
  const Size all{M, N, stages(K)};
  f.tiles = make_plan(&all, 1, nmat, split, cus);
  const int rest = (int)(M % 64);
  if (rest == 0 || rest > kSkinnyRows || M < 64) return f;
  const Size most{M - rest, N, all.nk};
  const Plan p = make_plan(&most, 1, nmat, split, cus);
  // A launch, and the weights once more at the rate that they stream from the last-level cache.
  if (p.time + 4.0 + (double)N * K * 2 * nmat / 4.0e6 < f.tiles.time) {
    f.rest = rest;
    f.tiles = p;
  }
  return f;
}

}  // namespace moe
