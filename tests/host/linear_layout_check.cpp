// Walks the loads of the dense projection's tiles on the host: for every stage, wavefront, lane and piece, what
// linear_layout.h's SourceMap addresses against what the staged tile needs.
#include <initializer_list>

#include "../../mixture_experts_layer_moe_amd/csrc/linear_layout.h"

namespace {

// Loads that go wrong over all tiles of an operand: one that lies in the resource must be the 16 bytes its place in LDS
// stands for, whole and inside the operand; one whose row or reduction index does not exist must lie outside.
template <bool COLS, int C, int NW, bool PAIRED>
int64_t walk(int64_t ld, int64_t extent, int64_t rows, int64_t R, int segments) {
  using namespace moe;
  const int64_t seg = (R + BK - 1) / BK;
  const int nk = (int)seg * segments;
  const int64_t size = 2 * (COLS ? (R - 1) * ld + extent : (extent - 1) * ld + R);  // bytes from first to last element
  constexpr int PIECES = C / (8 * NW), LPR = COLS ? C / 8 : 8;
  int64_t wrong = 0;
  for (int64_t c0 = 0; c0 < rows; c0 += C)
    for (int wave = 0; wave < NW; ++wave)
      for (int lane = 0; lane < 64; ++lane) {
        const SourceMap<COLS, C, NW, PAIRED> m(ld, extent, R, c0, (int)seg, nk, wave, lane);
        for (int kt = 0; kt < nk + 2; ++kt) {  // (loads run two stages ahead)
          const int64_t st = kt < nk ? kt % seg : kt;  // stage of its segment
          const int64_t base = 2 * (COLS ? c0 : c0 * ld) + st * m.adv;
          for (int p = 0; p < PIECES; ++p) {
            const int line = (p * NW + wave) * (64 / LPR) + lane / LPR;  // LDS row
            const int chunk = (lane % LPR) ^ (COLS ? swz_t<COLS ? C : 64>(line) : PAIRED ? swz_p(line) : swz(line));
            const int64_t row = COLS ? c0 + chunk * 8 : c0 + line, k = st * BK + (COLS ? line : chunk * 8);
            const bool need = kt < nk && row < extent && k < R;
            const uint32_t o = m.offset(kt) + p * m.step;
            const int64_t bytes = m.bytes(kt), at = base + o;
            const bool in = (int64_t)o < bytes;
            if (bytes < 0 || in != need) ++wrong;
            else if (in && (at != 2 * (COLS ? k * ld + row : row * ld + k) || (int64_t)o + 16 > bytes || at + 16 > size)) ++wrong;
          }
        }
      }
  return wrong;
}

}  // namespace

extern "C" {

// moe_linear's operands, x [M, K] and w [N, K], in the tiles of each kind (dual: two weight matrices).
int64_t forward_wrong(int64_t M, int64_t N, int64_t K) {
  return walk<false, 256, 8, false>(K, M, M, K, 1) + walk<false, 128, 4, false>(K, M, M, K, 1) +
         walk<false, 64, 4, false>(K, M, M, K, 1) + walk<false, 256, 8, true>(K, N, N, K, 1) +
         walk<false, 128, 8, true>(K, N, N, K, 1) + walk<false, 128, 4, true>(K, N, N, K, 1) +
         walk<false, 64, 8, true>(K, N, N, K, 1) + walk<false, 64, 4, true>(K, N, N, K, 1);
}

// moe_linear_backward's: dz [M, mats Np] as rows (input gradient) and as columns (weight gradients, the last matrix's),
// w [N, K] in `mats` segments and x [M, K] as columns.
int64_t backward_wrong(int64_t M, int64_t N, int64_t K, int mats) {
  const int64_t Np = (N + 63) / 64 * 64, ld = mats * Np;
  int64_t wrong = walk<false, 256, 8, false>(ld, M, M, ld, 1) + walk<false, 128, 4, false>(ld, M, M, ld, 1) +
                  walk<false, 64, 4, false>(ld, M, M, ld, 1);
  wrong += walk<true, 256, 8, false>(ld, Np, N, M, 1) + walk<true, 128, 4, false>(ld, Np, N, M, 1) + walk<true, 64, 4, false>(ld, Np, N, M, 1);
  for (int64_t R : {N, M})
    wrong += walk<true, 256, 8, false>(K, K, K, R, R == N ? mats : 1) + walk<true, 128, 8, false>(K, K, K, R, R == N ? mats : 1) +
             walk<true, 128, 4, false>(K, K, K, R, R == N ? mats : 1);
  return wrong;
}

// Tile kind, slices and streamed rows of moe_linear with a workspace on a device of 256 CUs.
void forward_tiles(int64_t M, int N, int K, int dual, int* out) {
  const moe::ForwardPlan f = moe::forward_plan(M, N, K, dual ? 2 : 1, true, 256);
  out[0] = f.tiles.kind;
  out[1] = f.tiles.S[0];
  out[2] = f.rest;
}

}  // extern "C"
