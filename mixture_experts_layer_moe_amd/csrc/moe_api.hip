// extern "C" entry points of libmoe.so: host-side validation, then launch.
// The operations and their argument conventions are documented in include/moe.h.
#include "../../include/moe.h"
#include "common.h"
#include "operators.h"

#include <math.h>

namespace {

constexpr int32_t kAbiVersion = 5;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool tile_m_ok(int32_t tm) { return tm == 16 || tm == 32 || tm == 64 || tm == 128 || tm == 256; }
// Bytes of an argument; absent ones overlap nothing.
struct Span {
  const void* p;
  size_t bytes;
};
bool overlap(const Span& a, const Span& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return a.p && b.p && x < y + b.bytes && y < x + a.bytes;
}
// Does one of the outputs overlap an input or another output?
template <int NO, int NI>
bool clash(const Span (&out)[NO], const Span (&in)[NI]) {
  for (int i = 0; i < NO; ++i) {
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return true;
    for (const Span& s : in)
      if (overlap(out[i], s)) return true;
  }
  return false;
}

moe_status launched(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH; }
int64_t min64(int64_t a, int64_t b) { return a < b ? a : b; }

}  // namespace

extern "C" {

const char* moe_status_str(int status) {
  switch (status) {
    case MOE_OK: return "MOE_OK";
    case MOE_ERR_INVALID_ARG: return "MOE_ERR_INVALID_ARG";
    case MOE_ERR_UNSUPPORTED: return "MOE_ERR_UNSUPPORTED";
    case MOE_ERR_WORKSPACE: return "MOE_ERR_WORKSPACE";
    case MOE_ERR_LAUNCH: return "MOE_ERR_LAUNCH";
    default: return "MOE_ERR_UNKNOWN";
  }
}

int32_t moe_abi_version(void) { return kAbiVersion; }

int64_t moe_rows_capacity(int64_t T, int32_t k, int32_t E_loc, int32_t tile_m) {
  if (T < 0 || k < 1 || E_loc < 1 || tile_m < 1) return -1;
  return T * min64(k, E_loc) + (int64_t)E_loc * (tile_m - 1);
}

int64_t moe_tiles_capacity(int64_t T, int32_t k, int32_t E_loc, int32_t tile_m) {
  if (T < 0 || k < 1 || E_loc < 1 || tile_m < 1) return -1;
  return T * min64(k, E_loc) / tile_m + E_loc;
}

size_t moe_permute_workspace_bytes(int64_t T, int32_t k, int32_t E_loc, int32_t num_ranks) {
  if (T < 0 || k < 1 || E_loc < 1 || num_ranks < 1) return 0;
  return moe::permute_ws_bytes(T, k, E_loc, num_ranks);
}

moe_status moe_route_topk(const float* logits, int64_t T, int32_t E, int32_t k, int32_t renormalize,
                          int32_t* topk_idx, float* topk_w, void* stream) {
  if (T < 0 || E < 1 || k < 1 || k > E) return MOE_ERR_INVALID_ARG;
  if (E > 1024 || k > 32) return MOE_ERR_UNSUPPORTED;
  if (T > (int64_t)INT32_MAX / 64) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!logits || !topk_idx || !topk_w) return MOE_ERR_INVALID_ARG;
  if (!aligned16(logits) || !aligned16(topk_idx) || !aligned16(topk_w)) return MOE_ERR_INVALID_ARG;
  return launched(moe::launch_route_topk(logits, T, E, k, renormalize, topk_idx, topk_w,
                                         static_cast<hipStream_t>(stream)));
}

}  // extern "C"

namespace {

// Shared validation and launch of moe_permute (caller's workspace) and
// moe_permute_noalloc (static == true: the library's fixed scratch).
moe_status permute_impl(const void* x, const int32_t* topk_idx, const int32_t* src_rank, int64_t T, int32_t H,
                        int32_t k, int32_t E, int32_t expert_begin, int32_t E_loc, int32_t num_ranks,
                        int32_t tile_m, void* x_perm, int32_t* expert_counts, int32_t* expert_offsets,
                        int32_t* row_src, int32_t* inv_perm, int32_t* tiles, int32_t* num_tiles, void* ws,
                        size_t ws_bytes, bool static_ws, void* stream) {
  if (T < 0 || H < 1 || k < 1 || E < 1 || k > E || E_loc < 1 || expert_begin < 0 ||
      (int64_t)expert_begin + E_loc > E || num_ranks < 1)
    return MOE_ERR_INVALID_ARG;
  if (H % 8 != 0 || !tile_m_ok(tile_m) || k > 32 || num_ranks > 64 || (int64_t)E_loc * num_ranks > 4096)
    return MOE_ERR_UNSUPPORTED;
  const int64_t R_cap = moe_rows_capacity(T, k, E_loc, tile_m);
  if (T * (int64_t)k > INT32_MAX || R_cap > INT32_MAX) return MOE_ERR_UNSUPPORTED;
  if (T > (1 << 26) - 16) return MOE_ERR_UNSUPPORTED;  // a wavefront a token: a grid holds fewer than 2^32 threads
  if (T == 0) return MOE_OK;
  // x and x_perm both null: indices only (the rows are gathered later by moe_grouped_ffn_gather).
  if ((x == nullptr) != (x_perm == nullptr)) return MOE_ERR_INVALID_ARG;
  if (x && (!aligned16(x) || !aligned16(x_perm))) return MOE_ERR_INVALID_ARG;
  const void* ptrs[] = {topk_idx, expert_counts, expert_offsets, row_src, inv_perm, tiles, num_tiles};
  for (const void* p : ptrs)
    if (!p || !aligned16(p)) return MOE_ERR_INVALID_ARG;
  if (src_rank && !aligned16(src_rank)) return MOE_ERR_INVALID_ARG;
  if (static_ws) {
    static_assert(moe::kPermuteStaticWsBytes == MOE_PERMUTE_NOALLOC_MAX_BYTES, "header and library agree");
    if (moe::permute_ws_bytes(T, k, E_loc, num_ranks) > moe::kPermuteStaticWsBytes) return MOE_ERR_WORKSPACE;
    if (moe::permute_static_ws(&ws) != hipSuccess) return MOE_ERR_LAUNCH;
  } else {
    if (!ws || !aligned16(ws)) return MOE_ERR_INVALID_ARG;
    if (ws_bytes < moe::permute_ws_bytes(T, k, E_loc, num_ranks)) return MOE_ERR_WORKSPACE;
  }
  moe::PermuteArgs a;
  a.x = static_cast<const uint16_t*>(x);
  a.topk_idx = topk_idx;
  a.src_rank = src_rank;
  a.T = T;
  a.H = H;
  a.k = k;
  a.E = E;
  a.expert_begin = expert_begin;
  a.E_loc = E_loc;
  a.num_ranks = src_rank ? num_ranks : 1;
  a.tile_m = tile_m;
  a.R_cap = R_cap;
  a.tiles_cap = moe_tiles_capacity(T, k, E_loc, tile_m);
  a.x_perm = static_cast<uint16_t*>(x_perm);
  a.counts = expert_counts;
  a.offsets = expert_offsets;
  a.row_src = row_src;
  a.inv_perm = inv_perm;
  a.tiles = tiles;
  a.num_tiles = num_tiles;
  a.ws = ws;
  return launched(moe::launch_permute(a, static_cast<hipStream_t>(stream)));
}

}  // namespace

extern "C" {

moe_status moe_permute(const void* x, const int32_t* topk_idx, const int32_t* src_rank, int64_t T, int32_t H,
                       int32_t k, int32_t E, int32_t expert_begin, int32_t E_loc, int32_t num_ranks,
                       int32_t tile_m, void* x_perm, int32_t* expert_counts, int32_t* expert_offsets,
                       int32_t* row_src, int32_t* inv_perm, int32_t* tiles, int32_t* num_tiles, void* ws,
                       size_t ws_bytes, void* stream) {
  return permute_impl(x, topk_idx, src_rank, T, H, k, E, expert_begin, E_loc, num_ranks, tile_m, x_perm,
                      expert_counts, expert_offsets, row_src, inv_perm, tiles, num_tiles, ws, ws_bytes, false,
                      stream);
}

moe_status moe_permute_noalloc(const void* x, const int32_t* topk_idx, const int32_t* src_rank, int64_t T,
                               int32_t H, int32_t k, int32_t E, int32_t expert_begin, int32_t E_loc,
                               int32_t num_ranks, int32_t tile_m, void* x_perm, int32_t* expert_counts,
                               int32_t* expert_offsets, int32_t* row_src, int32_t* inv_perm, int32_t* tiles,
                               int32_t* num_tiles, void* stream) {
  return permute_impl(x, topk_idx, src_rank, T, H, k, E, expert_begin, E_loc, num_ranks, tile_m, x_perm,
                      expert_counts, expert_offsets, row_src, inv_perm, tiles, num_tiles, nullptr, 0, true, stream);
}

size_t moe_grouped_ffn_workspace_bytes(int32_t tile_m, int32_t H) {
  if (!tile_m_ok(tile_m) || H < 1) return 0;
  return moe::grouped_ffn_ws_bytes(tile_m, H);
}

namespace {

// Shared validation and launch of moe_grouped_ffn (x_perm given) and
// moe_grouped_ffn_gather (x, row_src, T, k given, x_perm null).
moe_status grouped_ffn_impl(const void* x_perm, const void* x, const int32_t* row_src, int64_t T, int32_t k,
                            const int32_t* expert_counts, const int32_t* expert_offsets, const int32_t* tiles,
                            const int32_t* num_tiles, const void* w0, const void* w0_up, const void* w1,
                            int32_t E_loc, int32_t H, int32_t F, int32_t act, int32_t tile_m, int64_t R_cap,
                            int64_t tiles_cap, void* act_buf, float* y_perm, void* ws, size_t ws_bytes,
                            void* stream) {
  if (E_loc < 1 || H < 1 || F < 1 || R_cap < 0 || tiles_cap < 0) return MOE_ERR_INVALID_ARG;
  if (act != MOE_ACT_GELU && act != MOE_ACT_SWIGLU) return MOE_ERR_INVALID_ARG;
  if ((act == MOE_ACT_SWIGLU) != (w0_up != nullptr)) return MOE_ERR_INVALID_ARG;
  if (H % 128 != 0 || F % 128 != 0 || !tile_m_ok(tile_m)) return MOE_ERR_UNSUPPORTED;
  if (H > (1 << 20) || F > (1 << 20)) return MOE_ERR_UNSUPPORTED;  // 32-bit operand-panel offsets
  if (R_cap > INT32_MAX || tiles_cap > INT32_MAX / 2) return MOE_ERR_UNSUPPORTED;
  const bool gather = x_perm == nullptr;
  if (gather) {
    if (T < 0 || k < 1) return MOE_ERR_INVALID_ARG;
    if (T * (int64_t)H * 2 > INT32_MAX || T * (int64_t)k > INT32_MAX) return MOE_ERR_UNSUPPORTED;
  }
  if (R_cap == 0 || tiles_cap == 0 || (gather && T == 0)) return MOE_OK;
  const void* ptrs[] = {gather ? x : x_perm, expert_counts, expert_offsets, tiles, num_tiles, w0, w1, act_buf, y_perm};
  for (const void* p : ptrs)
    if (!p || !aligned16(p)) return MOE_ERR_INVALID_ARG;
  if (gather && (!row_src || !aligned16(row_src))) return MOE_ERR_INVALID_ARG;
  if (w0_up && !aligned16(w0_up)) return MOE_ERR_INVALID_ARG;
  if (ws) {
    if (!aligned16(ws)) return MOE_ERR_INVALID_ARG;
    if (ws_bytes < moe::grouped_ffn_ws_bytes(tile_m, H)) return MOE_ERR_WORKSPACE;
  }
  moe::FfnArgs a{};
  a.x_perm = static_cast<const uint16_t*>(x_perm);
  a.x = static_cast<const uint16_t*>(x);
  a.row_src = row_src;
  a.topk = k;
  a.T = T;
  a.counts = expert_counts;
  a.offsets = expert_offsets;
  a.tiles = tiles;
  a.num_tiles = num_tiles;
  a.w0 = static_cast<const uint16_t*>(w0);
  a.w0_up = static_cast<const uint16_t*>(w0_up);
  a.w1 = static_cast<const uint16_t*>(w1);
  a.E_loc = E_loc;
  a.H = H;
  a.F = F;
  a.act = act;
  a.tile_m = tile_m;
  a.R_cap = R_cap;
  a.tiles_cap = tiles_cap;
  a.act_buf = static_cast<uint16_t*>(act_buf);
  a.y_perm = y_perm;
  a.ws = ws;
  a.stream = static_cast<hipStream_t>(stream);
  return launched(moe::launch_grouped_ffn(a));
}

}  // namespace

moe_status moe_grouped_ffn(const void* x_perm, const int32_t* expert_counts, const int32_t* expert_offsets,
                           const int32_t* tiles, const int32_t* num_tiles, const void* w0, const void* w0_up,
                           const void* w1, int32_t E_loc, int32_t H, int32_t F, int32_t act, int32_t tile_m,
                           int64_t R_cap, int64_t tiles_cap, void* act_buf, float* y_perm, void* ws,
                           size_t ws_bytes, void* stream) {
  if (!x_perm) return MOE_ERR_INVALID_ARG;
  return grouped_ffn_impl(x_perm, nullptr, nullptr, 0, 0, expert_counts, expert_offsets, tiles, num_tiles, w0, w0_up,
                          w1, E_loc, H, F, act, tile_m, R_cap, tiles_cap, act_buf, y_perm, ws, ws_bytes, stream);
}

moe_status moe_grouped_ffn_gather(const void* x, const int32_t* row_src, int64_t T, int32_t k,
                                  const int32_t* expert_counts, const int32_t* expert_offsets,
                                  const int32_t* tiles, const int32_t* num_tiles, const void* w0,
                                  const void* w0_up, const void* w1, int32_t E_loc, int32_t H, int32_t F,
                                  int32_t act, int32_t tile_m, int64_t R_cap, int64_t tiles_cap, void* act_buf,
                                  float* y_perm, void* ws, size_t ws_bytes, void* stream) {
  if (!x && T != 0) return MOE_ERR_INVALID_ARG;
  return grouped_ffn_impl(nullptr, x, row_src, T, k, expert_counts, expert_offsets, tiles, num_tiles, w0, w0_up, w1,
                          E_loc, H, F, act, tile_m, R_cap, tiles_cap, act_buf, y_perm, ws, ws_bytes, stream);
}

size_t moe_ffn_combine_fused_workspace_bytes(int64_t tiles_cap, int32_t H) {
  if (tiles_cap < 0 || H < 256 || H % 256 != 0 || tiles_cap > INT32_MAX / 2) return 0;
  return moe::fused_ffn_ws_bytes(tiles_cap, H);
}

moe_status moe_ffn_combine_fused(const void* x_perm, const int32_t* expert_counts, const int32_t* expert_offsets,
                                 const int32_t* tiles, const int32_t* num_tiles, const void* w0, const void* w0_up,
                                 const void* w1, int32_t E_loc, int32_t H, int32_t F, int32_t act, int32_t tile_m,
                                 int64_t R_cap, int64_t tiles_cap, void* act_buf, float* y_perm,
                                 const int32_t* inv_perm, const float* topk_w, int64_t T, int32_t k, float* out,
                                 void* ws, size_t ws_bytes, void* stream) {
  if (E_loc < 1 || H < 1 || F < 1 || R_cap < 0 || tiles_cap < 0 || T < 0 || k < 1) return MOE_ERR_INVALID_ARG;
  if (act != MOE_ACT_GELU && act != MOE_ACT_SWIGLU) return MOE_ERR_INVALID_ARG;
  if ((act == MOE_ACT_SWIGLU) != (w0_up != nullptr)) return MOE_ERR_INVALID_ARG;
  if (tile_m != 256 || H % 256 != 0 || F % 128 != 0) return MOE_ERR_UNSUPPORTED;
  if (H > (1 << 20) || F > (1 << 20) || k > 32) return MOE_ERR_UNSUPPORTED;
  if (R_cap > INT32_MAX || tiles_cap > INT32_MAX / 2 || T > INT32_MAX) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  const void* ptrs[] = {x_perm, expert_counts, expert_offsets, tiles, num_tiles, w0, w1, act_buf, y_perm,
                        inv_perm, topk_w, out, ws};
  for (const void* p : ptrs)
    if (!p || !aligned16(p)) return MOE_ERR_INVALID_ARG;
  if (w0_up && !aligned16(w0_up)) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < moe::fused_ffn_ws_bytes(tiles_cap, H)) return MOE_ERR_WORKSPACE;
  moe::FfnArgs a{};
  a.x_perm = static_cast<const uint16_t*>(x_perm);
  a.counts = expert_counts;
  a.offsets = expert_offsets;
  a.tiles = tiles;
  a.num_tiles = num_tiles;
  a.w0 = static_cast<const uint16_t*>(w0);
  a.w0_up = static_cast<const uint16_t*>(w0_up);
  a.w1 = static_cast<const uint16_t*>(w1);
  a.E_loc = E_loc;
  a.H = H;
  a.F = F;
  a.act = act;
  a.tile_m = tile_m;
  a.R_cap = R_cap;
  a.tiles_cap = tiles_cap;
  a.act_buf = static_cast<uint16_t*>(act_buf);
  a.y_perm = y_perm;
  a.ws = ws;
  a.topk = k;
  a.T = T;
  a.stream = static_cast<hipStream_t>(stream);
  return launched(moe::launch_ffn_fused(a, inv_perm, topk_w, out));
}

moe_status moe_combine(const float* y_perm, const int32_t* inv_perm, const float* topk_w, int64_t T, int32_t k,
                       int32_t H, int64_t R_cap, float* out, void* stream) {
  if (T < 0 || k < 1 || H < 1 || R_cap < 0) return MOE_ERR_INVALID_ARG;
  if (H % 4 != 0 || k > 32 || T > INT32_MAX) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!y_perm || !inv_perm || !topk_w || !out) return MOE_ERR_INVALID_ARG;
  if (!aligned16(y_perm) || !aligned16(inv_perm) || !aligned16(topk_w) || !aligned16(out))
    return MOE_ERR_INVALID_ARG;
  return launched(moe::launch_combine(y_perm, inv_perm, topk_w, T, k, H, R_cap, out,
                                      static_cast<hipStream_t>(stream)));
}

moe_status moe_route_grouped(const float* logits, const float* bias, int64_t T, int32_t E, int32_t k, int32_t score,
                             int32_t n_group, int32_t topk_group, int32_t group_top, int32_t renormalize, float scale,
                             int32_t* topk_idx, float* topk_w, void* stream) {
  if (T < 0 || E < 1 || k < 1 || k > E || !isfinite(scale)) return MOE_ERR_INVALID_ARG;
  if (score != MOE_SCORE_SOFTMAX && score != MOE_SCORE_SIGMOID) return MOE_ERR_INVALID_ARG;
  if (n_group < 1 || n_group > E || E % n_group != 0 || topk_group < 1 || topk_group > n_group)
    return MOE_ERR_INVALID_ARG;
  if (group_top < 1 || group_top > 2 || group_top > E / n_group || (int64_t)k > (int64_t)topk_group * (E / n_group))
    return MOE_ERR_INVALID_ARG;
  if (E > 1024 || k > 32 || n_group > 64 || T > (int64_t)INT32_MAX / 64) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!logits || !topk_idx || !topk_w) return MOE_ERR_INVALID_ARG;
  if (!aligned16(logits) || !aligned16(bias) || !aligned16(topk_idx) || !aligned16(topk_w)) return MOE_ERR_INVALID_ARG;
  const size_t e = (size_t)E * 4, te = (size_t)T * e, tk = (size_t)T * k * 4;
  const Span outs[] = {{topk_idx, tk}, {topk_w, tk}}, ins[] = {{logits, te}, {bias, e}};
  if (clash(outs, ins)) return MOE_ERR_INVALID_ARG;
  const moe::RouteArgs a{logits,  bias,       T,         E,     k,        score == MOE_SCORE_SIGMOID, renormalize != 0,
                         n_group, topk_group, group_top, scale, topk_idx, topk_w};
  return launched(moe::launch_route_grouped(a, static_cast<hipStream_t>(stream)));
}

moe_status moe_route_grouped_bias_backward(const float* logits, const float* bias, const int32_t* topk_idx,
                                           const float* d_topk_w, int64_t T, int32_t E, int32_t k, int32_t score,
                                           int32_t renormalize, float scale, float* d_logits, void* stream) {
  if (T < 0 || E < 1 || k < 1 || k > E || !isfinite(scale)) return MOE_ERR_INVALID_ARG;
  if (score != MOE_SCORE_SOFTMAX && score != MOE_SCORE_SIGMOID) return MOE_ERR_INVALID_ARG;
  if (E > 1024 || k > 32 || T > (int64_t)INT32_MAX / 64) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  const void* ptrs[] = {logits, topk_idx, d_topk_w, d_logits};
  for (const void* p : ptrs)
    if (!p || !aligned16(p)) return MOE_ERR_INVALID_ARG;
  if (!aligned16(bias)) return MOE_ERR_INVALID_ARG;
  const size_t te = (size_t)T * E * 4, tk = (size_t)T * k * 4;
  const Span outs[] = {{d_logits, te}}, ins[] = {{logits, te}, {bias, (size_t)E * 4}, {topk_idx, tk}, {d_topk_w, tk}};
  if (clash(outs, ins)) return MOE_ERR_INVALID_ARG;
  const moe::RouteBwdArgs a{logits, bias, topk_idx, d_topk_w, T, E, k, score == MOE_SCORE_SIGMOID, renormalize != 0,
                            scale, d_logits};
  return launched(moe::launch_route_grouped_backward(a, static_cast<hipStream_t>(stream)));
}

moe_status moe_route_grouped_backward(const float* logits, const int32_t* topk_idx, const float* d_topk_w, int64_t T,
                                      int32_t E, int32_t k, int32_t score, int32_t renormalize, float scale,
                                      float* d_logits, void* stream) {
  return moe_route_grouped_bias_backward(logits, nullptr, topk_idx, d_topk_w, T, E, k, score, renormalize, scale,
                                         d_logits, stream);
}

moe_status moe_combine_backward(const float* d_out, const float* y_perm, const int32_t* inv_perm, const float* topk_w,
                                int64_t T, int32_t k, int32_t H, int64_t R_cap, float* d_y_perm, float* d_topk_w,
                                void* stream) {
  if (T < 0 || k < 1 || H < 1 || R_cap < 0) return MOE_ERR_INVALID_ARG;
  if (H % 4 != 0 || k > 32 || T > INT32_MAX) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  const void* ptrs[] = {d_out, y_perm, inv_perm, topk_w, d_y_perm, d_topk_w};
  for (const void* p : ptrs)
    if (!p || !aligned16(p)) return MOE_ERR_INVALID_ARG;
  const size_t th = (size_t)T * H * 4, rh = (size_t)R_cap * H * 4, tk = (size_t)T * k * 4;
  const Span outs[] = {{d_y_perm, rh}, {d_topk_w, tk}}, ins[] = {{d_out, th}, {y_perm, rh}, {inv_perm, tk}, {topk_w, tk}};
  if (clash(outs, ins)) return MOE_ERR_INVALID_ARG;
  return launched(moe::launch_combine_backward(d_out, y_perm, inv_perm, topk_w, T, k, H, R_cap, d_y_perm, d_topk_w,
                                               static_cast<hipStream_t>(stream)));
}

}  // extern "C"

namespace {

bool act_ok(int32_t act) {
  return act == MOE_ACT_GELU || act == MOE_ACT_SWIGLU || act == MOE_ACT_NONE || act == MOE_ACT_SILU;
}

// Sizes of moe_linear and moe_linear_backward.
moe_status linear_sizes(int64_t M, int32_t N, int32_t K, int32_t act) {
  if (M < 0 || N < 1 || K < 1 || !act_ok(act)) return MOE_ERR_INVALID_ARG;
  if (K % 8 != 0 || N > (1 << 20) || K > (1 << 20) || M > INT32_MAX) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// hipErrorNotSupported: a product of more tiles than a launch takes, found before anything is enqueued.
moe_status linear_launched(hipError_t e) { return e == hipErrorNotSupported ? MOE_ERR_UNSUPPORTED : launched(e); }

}  // namespace

extern "C" {

size_t moe_linear_workspace_bytes(int64_t M, int32_t N, int32_t K, int32_t act) {
  if (linear_sizes(M, N, K, act) != MOE_OK) return 0;
  return moe::linear_ws_bytes(M, N, K, act);
}

moe_status moe_linear(const void* x, const void* w, const void* w_up, const float* bias, const float* bias_up,
                      const void* residual, int64_t M, int32_t N, int32_t K, int32_t act, int32_t out_dtype, void* z,
                      void* z_up, void* out, void* ws, size_t ws_bytes, void* stream) {
  const moe_status st = linear_sizes(M, N, K, act);
  if (st != MOE_OK) return st;
  if (out_dtype != MOE_BF16 && out_dtype != MOE_F32) return MOE_ERR_INVALID_ARG;
  const bool dual = act == MOE_ACT_SWIGLU;
  if (!dual && (w_up || bias_up || z_up)) return MOE_ERR_INVALID_ARG;
  if (M == 0) return MOE_OK;
  if (!x || !w || !out || (dual && !w_up)) return MOE_ERR_INVALID_ARG;
  const void* ptrs[] = {x, w, w_up, bias, bias_up, residual, z, z_up, out, ws};
  for (const void* p : ptrs)
    if (!aligned16(p)) return MOE_ERR_INVALID_ARG;
  if (ws && ws_bytes < moe::linear_ws_bytes(M, N, K, act)) return MOE_ERR_WORKSPACE;
  const size_t mn = (size_t)M * N, nk = (size_t)N * K * 2, nb = (size_t)N * 4, es = out_dtype == MOE_F32 ? 4 : 2;
  const Span outs[] = {{out, mn * es}, {z, mn * 2}, {z_up, mn * 2}, {ws, ws_bytes}};
  const Span ins[] = {{x, (size_t)M * K * 2}, {w, nk}, {w_up, nk}, {bias, nb}, {bias_up, nb},
                      {residual == out ? nullptr : residual, mn * es}};
  if (clash(outs, ins)) return MOE_ERR_INVALID_ARG;
  moe::LinearArgs a{};
  a.x = static_cast<const uint16_t*>(x);
  a.w = static_cast<const uint16_t*>(w);
  a.w_up = static_cast<const uint16_t*>(w_up);
  a.bias = bias;
  a.bias_up = bias_up;
  a.residual = residual;
  a.M = M;
  a.N = N;
  a.K = K;
  a.act = act;
  a.out_f32 = out_dtype == MOE_F32;
  a.z = static_cast<uint16_t*>(z);
  a.z_up = static_cast<uint16_t*>(z_up);
  a.out = out;
  a.ws = ws;
  return linear_launched(moe::launch_linear(a, static_cast<hipStream_t>(stream)));
}

size_t moe_linear_backward_workspace_bytes(int64_t M, int32_t N, int32_t K, int32_t act) {
  if (linear_sizes(M, N, K, act) != MOE_OK) return 0;
  return moe::linear_backward_ws_bytes(M, N, K, act);
}

moe_status moe_linear_backward(const void* d_out, const void* x, const void* w, const void* w_up, const void* z,
                               const void* z_up, int64_t M, int32_t N, int32_t K, int32_t act, int32_t out_dtype,
                               void* d_x, void* d_w, void* d_w_up, float* d_bias, float* d_bias_up, void* ws,
                               size_t ws_bytes, void* stream) {
  const moe_status st = linear_sizes(M, N, K, act);
  if (st != MOE_OK) return st;
  if (out_dtype != MOE_BF16 && out_dtype != MOE_F32) return MOE_ERR_INVALID_ARG;
  const bool dual = act == MOE_ACT_SWIGLU;
  if (!dual && (w_up || z_up || d_w_up || d_bias_up)) return MOE_ERR_INVALID_ARG;
  if (act == MOE_ACT_NONE && z) return MOE_ERR_INVALID_ARG;
  const void* ptrs[] = {d_out, x, w, w_up, z, z_up, d_x, d_w, d_w_up, d_bias, d_bias_up, ws};
  for (const void* p : ptrs)
    if (!aligned16(p)) return MOE_ERR_INVALID_ARG;
  if (M > 0) {
    if (!d_out || !ws || (act != MOE_ACT_NONE && !z) || (dual && !z_up)) return MOE_ERR_INVALID_ARG;
    if (d_x && (!w || (dual && !w_up))) return MOE_ERR_INVALID_ARG;
    if ((d_w || d_w_up) && !x) return MOE_ERR_INVALID_ARG;
    if (ws_bytes < moe::linear_backward_ws_bytes(M, N, K, act)) return MOE_ERR_WORKSPACE;
    const size_t mn = (size_t)M * N, mk = (size_t)M * K * 2, nk = (size_t)N * K * 2, nb = (size_t)N * 4;
    const Span outs[] = {{d_x, mk}, {d_w, nk}, {d_w_up, nk}, {d_bias, nb}, {d_bias_up, nb}, {ws, ws_bytes}};
    const Span ins[] = {{d_out, mn * (out_dtype == MOE_F32 ? 4 : 2)}, {x, mk}, {w, nk}, {w_up, nk}, {z, mn * 2}, {z_up, mn * 2}};
    if (clash(outs, ins)) return MOE_ERR_INVALID_ARG;
  }
  moe::LinearBwdArgs a{};
  a.d_out = d_out;
  a.x = static_cast<const uint16_t*>(x);
  a.w = static_cast<const uint16_t*>(w);
  a.w_up = static_cast<const uint16_t*>(w_up);
  a.z = static_cast<const uint16_t*>(z);
  a.z_up = static_cast<const uint16_t*>(z_up);
  a.M = M;
  a.N = N;
  a.K = K;
  a.act = act;
  a.out_f32 = out_dtype == MOE_F32;
  a.d_x = static_cast<uint16_t*>(d_x);
  a.d_w = static_cast<uint16_t*>(d_w);
  a.d_w_up = static_cast<uint16_t*>(d_w_up);
  a.d_bias = d_bias;
  a.d_bias_up = d_bias_up;
  a.ws = ws;
  return linear_launched(moe::launch_linear_backward(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

namespace {

// Sizes of the products of MXFP4 operands, but for the rows.
moe_status mxfp4_sizes(int32_t N, int32_t K, int32_t act) {
  if (N < 1 || K < 1 || !act_ok(act)) return MOE_ERR_INVALID_ARG;
  if (K % 128 != 0 || N > (1 << 20) || K > (1 << 20)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

moe_status mxfp4_blocks(int64_t R, int32_t K, int32_t dtype) {
  if (R < 0 || K < 1 || (dtype != MOE_BF16 && dtype != MOE_F32)) return MOE_ERR_INVALID_ARG;
  if (K % 32 != 0 || R > ((int64_t)1 << 36) / K) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

}  // namespace

extern "C" {

moe_status moe_mxfp4_quantize(const void* x, int64_t R, int32_t K, int32_t x_dtype, void* codes, void* scales,
                              void* stream) {
  const moe_status st = mxfp4_blocks(R, K, x_dtype);
  if (st != MOE_OK || R == 0) return st;
  if (!x || !codes || !scales || !aligned16(x) || !aligned16(codes) || !aligned16(scales)) return MOE_ERR_INVALID_ARG;
  const size_t n = (size_t)R * K;
  const Span outs[] = {{codes, n / 2}, {scales, n / 32}}, ins[] = {{x, n * (x_dtype == MOE_F32 ? 4 : 2)}};
  if (clash(outs, ins)) return MOE_ERR_INVALID_ARG;
  return launched(moe::launch_mxfp4_quantize(x, x_dtype == MOE_F32, R * (K / 32), static_cast<uint8_t*>(codes),
                                             static_cast<uint8_t*>(scales), static_cast<hipStream_t>(stream)));
}

moe_status moe_mxfp4_dequantize(const void* codes, const void* scales, int64_t R, int32_t K, int32_t out_dtype, void* out,
                                void* stream) {
  const moe_status st = mxfp4_blocks(R, K, out_dtype);
  if (st != MOE_OK || R == 0) return st;
  if (!out || !codes || !scales || !aligned16(out) || !aligned16(codes) || !aligned16(scales)) return MOE_ERR_INVALID_ARG;
  const size_t n = (size_t)R * K;
  const Span outs[] = {{out, n * (out_dtype == MOE_F32 ? 4 : 2)}}, ins[] = {{codes, n / 2}, {scales, n / 32}};
  if (clash(outs, ins)) return MOE_ERR_INVALID_ARG;
  return linear_launched(moe::launch_mxfp4_dequantize(static_cast<const uint8_t*>(codes), static_cast<const uint8_t*>(scales),
                                                      R * (K / 32), out_dtype == MOE_F32, out, static_cast<hipStream_t>(stream)));
}

// (no size splits its reduction, so none needs a buffer; moe_linear_mxfp4 checks the one it is given)
size_t moe_linear_mxfp4_workspace_bytes(int64_t, int32_t, int32_t, int32_t) { return 0; }

moe_status moe_linear_mxfp4(const void* x_codes, const void* x_scales, const void* w_codes, const void* w_scales,
                            const void* w_up_codes, const void* w_up_scales, const float* bias, const float* bias_up,
                            const void* residual, int64_t M, int32_t N, int32_t K, int32_t act, int32_t out_dtype, void* out,
                            void* ws, size_t ws_bytes, void* stream) {
  if (M < 0 || (out_dtype != MOE_BF16 && out_dtype != MOE_F32)) return MOE_ERR_INVALID_ARG;
  const moe_status st = mxfp4_sizes(N, K, act);
  if (st != MOE_OK) return st;
  if (M > INT32_MAX) return MOE_ERR_UNSUPPORTED;
  const bool dual = act == MOE_ACT_SWIGLU;
  if (!dual && (w_up_codes || w_up_scales || bias_up)) return MOE_ERR_INVALID_ARG;
  if (M == 0) return MOE_OK;
  if (!x_codes || !x_scales || !w_codes || !w_scales || !out || (dual && (!w_up_codes || !w_up_scales)))
    return MOE_ERR_INVALID_ARG;
  const void* ptrs[] = {x_codes, x_scales, w_codes, w_scales, w_up_codes, w_up_scales, bias, bias_up, residual, out, ws};
  for (const void* p : ptrs)
    if (!aligned16(p)) return MOE_ERR_INVALID_ARG;
  const size_t mn = (size_t)M * N * (out_dtype == MOE_F32 ? 4 : 2), mk = (size_t)M * K, nk = (size_t)N * K, nb = (size_t)N * 4;
  const Span outs[] = {{out, mn}, {ws, ws_bytes}};
  const Span ins[] = {{x_codes, mk / 2}, {x_scales, mk / 32}, {w_codes, nk / 2}, {w_scales, nk / 32}, {w_up_codes, nk / 2},
                      {w_up_scales, nk / 32}, {bias, nb}, {bias_up, nb}, {residual == out ? nullptr : residual, mn}};
  if (clash(outs, ins)) return MOE_ERR_INVALID_ARG;
  moe::MxLinearArgs a{};
  a.x = {static_cast<const uint8_t*>(x_codes), static_cast<const uint8_t*>(x_scales)};
  a.w = {static_cast<const uint8_t*>(w_codes), static_cast<const uint8_t*>(w_scales)};
  a.w_up = {static_cast<const uint8_t*>(w_up_codes), static_cast<const uint8_t*>(w_up_scales)};
  a.bias = bias;
  a.bias_up = bias_up;
  a.residual = residual;
  a.M = M;
  a.N = N;
  a.K = K;
  a.act = act;
  a.out_f32 = out_dtype == MOE_F32;
  a.out = out;
  return linear_launched(moe::launch_linear_mxfp4(a, static_cast<hipStream_t>(stream)));
}

moe_status moe_grouped_linear_mxfp4(const void* x_codes, const void* x_scales, const int32_t* row_src, int64_t T, int32_t k,
                                    const int32_t* expert_counts, const int32_t* expert_offsets, const int32_t* tiles,
                                    const int32_t* num_tiles, const void* w_codes, const void* w_scales,
                                    const void* w_up_codes, const void* w_up_scales, int32_t E_loc, int32_t N, int32_t K,
                                    int32_t act, int32_t tile_m, int64_t R_cap, int64_t tiles_cap, int32_t out_dtype,
                                    void* out, void* stream) {
  if (E_loc < 1 || R_cap < 0 || tiles_cap < 0 || (out_dtype != MOE_BF16 && out_dtype != MOE_F32)) return MOE_ERR_INVALID_ARG;
  if (row_src && (T < 0 || k < 1)) return MOE_ERR_INVALID_ARG;
  const moe_status st = mxfp4_sizes(N, K, act);
  if (st != MOE_OK) return st;
  if (!tile_m_ok(tile_m) || R_cap > INT32_MAX || tiles_cap > INT32_MAX / 32) return MOE_ERR_UNSUPPORTED;
  if (row_src && (k > 32 || T > (int64_t)INT32_MAX / (K / 2))) return MOE_ERR_UNSUPPORTED;
  const bool dual = act == MOE_ACT_SWIGLU;
  if (!dual && (w_up_codes || w_up_scales)) return MOE_ERR_INVALID_ARG;
  if (R_cap == 0 || tiles_cap == 0 || (row_src && T == 0)) return MOE_OK;
  const void* ptrs[] = {x_codes, x_scales, expert_counts, expert_offsets, tiles, num_tiles, w_codes, w_scales, out};
  for (const void* p : ptrs)
    if (!p || !aligned16(p)) return MOE_ERR_INVALID_ARG;
  if (!aligned16(row_src) || !aligned16(w_up_codes) || !aligned16(w_up_scales)) return MOE_ERR_INVALID_ARG;
  if (dual && (!w_up_codes || !w_up_scales)) return MOE_ERR_INVALID_ARG;
  const size_t xk = (size_t)(row_src ? T : R_cap) * K, nk = (size_t)E_loc * N * K, e4 = (size_t)E_loc * 4;
  const Span outs[] = {{out, (size_t)R_cap * N * (out_dtype == MOE_F32 ? 4 : 2)}};
  const Span ins[] = {{x_codes, xk / 2}, {x_scales, xk / 32}, {row_src, (size_t)R_cap * 4}, {expert_counts, e4},
                      {expert_offsets, e4 + 4}, {tiles, (size_t)tiles_cap * 8}, {num_tiles, 4}, {w_codes, nk / 2},
                      {w_scales, nk / 32}, {w_up_codes, nk / 2}, {w_up_scales, nk / 32}};
  if (clash(outs, ins)) return MOE_ERR_INVALID_ARG;
  moe::MxLinearArgs a{};
  a.x = {static_cast<const uint8_t*>(x_codes), static_cast<const uint8_t*>(x_scales)};
  a.w = {static_cast<const uint8_t*>(w_codes), static_cast<const uint8_t*>(w_scales)};
  a.w_up = {static_cast<const uint8_t*>(w_up_codes), static_cast<const uint8_t*>(w_up_scales)};
  a.M = row_src ? T : R_cap;
  a.N = N;
  a.K = K;
  a.act = act;
  a.out_f32 = out_dtype == MOE_F32;
  a.out = out;
  a.counts = expert_counts;
  a.offsets = expert_offsets;
  a.tiles = tiles;
  a.num_tiles = num_tiles;
  a.row_src = row_src;
  a.topk = k;
  a.tile_m = tile_m;
  a.E_loc = E_loc;
  a.tiles_cap = tiles_cap;
  a.R_cap = R_cap;
  return linear_launched(moe::launch_grouped_linear_mxfp4(a, static_cast<hipStream_t>(stream)));
}

size_t moe_few_tokens_workspace_bytes(int64_t T, int32_t k, int32_t F) {
  if (T < 1 || T > moe::kFewTokens || k < 1 || k > 32 || F < 1 || F > (1 << 20)) return 0;
  return moe::few_tokens_ws_bytes((int)T, k, F);
}

moe_status moe_few_tokens(const void* x, const float* logits, int64_t T, int32_t E, int32_t k, int32_t renormalize,
                          int32_t expert_begin, int32_t E_loc, const void* w0, const void* w0_scales, const void* w0_up,
                          const void* w0_up_scales, const void* w1, const void* w1_scales, int32_t H, int32_t F, int32_t act,
                          int32_t* topk_idx, float* topk_w, float* out, void* ws, size_t ws_bytes, void* stream) {
  if (T < 0 || E < 1 || k < 1 || k > E || E_loc < 1 || expert_begin < 0 || (int64_t)expert_begin + E_loc > E || H < 1 || F < 1)
    return MOE_ERR_INVALID_ARG;
  if (act != MOE_ACT_GELU && act != MOE_ACT_SWIGLU) return MOE_ERR_INVALID_ARG;
  const bool dual = act == MOE_ACT_SWIGLU, mx = w0_scales != nullptr;
  if (!dual && (w0_up || w0_up_scales)) return MOE_ERR_INVALID_ARG;
  if ((w1_scales != nullptr) != mx || (dual && (w0_up_scales != nullptr) != mx)) return MOE_ERR_INVALID_ARG;
  if (T > moe::kFewTokens || E > 1024 || k > 32 || H % 128 != 0 || F % 128 != 0 || H > (1 << 20) || F > (1 << 20))
    return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  const void* ptrs[] = {x, w0, w1, topk_idx, topk_w, out, ws};
  for (const void* p : ptrs)
    if (!p || !aligned16(p)) return MOE_ERR_INVALID_ARG;
  if ((dual && !w0_up) || !aligned16(w0_up) || !aligned16(logits) || !aligned16(w0_scales) || !aligned16(w0_up_scales) ||
      !aligned16(w1_scales))
    return MOE_ERR_INVALID_ARG;
  if (ws_bytes < moe::few_tokens_ws_bytes((int)T, k, F)) return MOE_ERR_WORKSPACE;
  const size_t n = (size_t)E_loc * F * H, wb = mx ? n / 2 : n * 2, tk = (size_t)T * k * 4;
  const Span ins[] = {{x, (size_t)T * H * 2}, {logits, (size_t)T * E * 4}, {w0, wb}, {w0_up, wb}, {w1, wb},
                      {w0_scales, n / 32}, {w0_up_scales, n / 32}, {w1_scales, n / 32}};
  const Span outs[] = {{out, (size_t)T * H * 4}, {ws, ws_bytes}, {topk_idx, tk}, {topk_w, tk}};
  if (clash(outs, ins)) return MOE_ERR_INVALID_ARG;
  const moe::FewArgs a{static_cast<const uint16_t*>(x), logits, (int)T, E, k, expert_begin, E_loc, H, F, renormalize != 0,
                       w0, w0_up, w1, static_cast<const uint8_t*>(w0_scales), static_cast<const uint8_t*>(w0_up_scales),
                       static_cast<const uint8_t*>(w1_scales), topk_idx, topk_w, out, ws};
  return launched(moe::launch_few_tokens(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
