// Where the loads of the dense projection's tiles lie: integer arithmetic alone, so that a host test can walk every
// lane of every stage through it.
#pragma once

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

}  // namespace moe
