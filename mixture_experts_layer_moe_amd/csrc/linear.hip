// Dense projection with bias, activation and residual in its epilogue, and its
// gradients.
//
//   forward   z = x . w^T + b;  out = act(z) [* (x . w_up^T + b_up)] + residual
//   backward  dz = d_out * act'(z);  d_x = dz . w;  d_w = dz^T . x;  d_b = sum over the rows of dz
//
// All three products run on one tile scheme, C[m, n] = sum_r A(m, r) * B(n, r)
// with v_mfma_f32_32x32x16_bf16 and fp32 accumulators.  An operand is stored
// either with the reduction index contiguous (rows: x and w in the forward
// product, dz in d_x) or with it outermost (columns: w in d_x, dz and x in
// d_w).  Rows are staged in LDS as 128-byte lines of 64 reduction indices and
// read 16 bytes a lane; columns are staged as stored, 64 reduction indices of
// BM or BN columns, and read with the transposing LDS read (ds_read_b64_tr_b16:
// the 16 lanes of a group, reading 4 rows of 16 columns, each get one column),
// so no operand is transposed in memory.
#include "operators.h"

#include <float.h>

namespace moe {
namespace {

constexpr int BK = 64;  // reduction indices per stage

typedef __attribute__((__vector_size__(16 * sizeof(float)))) float floatx16;
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
// Rows operand: LDS row of 128 B per operand row, 16-byte chunk index XORed with swz(row) so that
// consecutive lanes (rows) at one chunk hit distinct banks.
__device__ __forceinline__ int swz(int row) { return (row & 7) ^ ((row >> 3) & 1); }
// Columns operand of C columns: LDS row of 2 C bytes per reduction index; a transposing read covers 4
// consecutive rows of a 64-byte column span per half wavefront, so the 64-byte unit is XORed with the row to
// spread those over all 64 banks.
template <int C>
__device__ __forceinline__ int swz_t(int r) {
  return C >= 128 ? (r & 3) << 2 : ((r >> 1) & 1) << 2;
}

// MFMA fragment (32 operand rows from row c0, 16 reduction indices from 16 ks) of a staged operand: lane holds
// row c0 + lane % 32, reduction indices 16 ks + 8 (lane / 32) + 0..7.
template <bool COLS, int C>
__device__ __forceinline__ bf16x8 fragment(const char* tile, int c0, int ks, int lane) {
  if constexpr (!COLS) {
    const int row = c0 + (lane & 31), chunk = ks * 2 + (lane >> 5);
    return *reinterpret_cast<const bf16x8*>(tile + row * 128 + ((chunk ^ swz(row)) << 4));
  } else {
    const int l16 = lane & 15;
    const int r = ks * 16 + 8 * (lane >> 5) + (l16 >> 2);
    const int chunk = (c0 >> 3) + 2 * ((lane >> 4) & 1) + ((l16 & 3) >> 1);
    const char* p = tile + r * (2 * C) + ((chunk ^ swz_t<C>(r)) << 4) + (l16 & 1) * 8;
    typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
    struct { s16x4 lo, hi; } f;
    f.lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
    f.hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 4 * (2 * C)));  // rows r + 4: same swizzle
    return __builtin_bit_cast(bf16x8, f);
  }
}

struct Operand {
  const uint16_t* p;  // first element
  int64_t ld;         // elements between rows (stored rows)
  int64_t rows;       // operand rows (m or n); columns operand: columns that may be read
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

// Four consecutive outputs of one row, the first of them column n (a multiple of 4) of N.
__device__ __forceinline__ void store4(const Epilogue& e, int64_t row, int n, int N, const float (&g)[4],
                                       const float (&u)[4]) {
  const bool dual = e.act == ACT_SWIGLU;
  const int64_t at = row * N + n;
  const int cnt = N - n < 4 ? N - n : 4;
  const bool vec = (N & 3) == 0;  // then the row's 4-element groups are aligned
  float v[4], a[4], b[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const bool in = q < cnt;
    a[q] = g[q] + (e.bias && in ? e.bias[n + q] : 0.f);
    b[q] = u[q] + (e.bias_up && in ? e.bias_up[n + q] : 0.f);
    v[q] = activate(e.act, a[q]) * (dual ? b[q] : 1.f);
  }
  auto put = [&](uint16_t* o, const float (&x)[4]) {
    uint16_t h[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) h[q] = f2bf_bits(x[q]);
    if (vec) {
      *reinterpret_cast<uint2*>(o + at) =
          uint2{(uint32_t)h[0] | ((uint32_t)h[1] << 16), (uint32_t)h[2] | ((uint32_t)h[3] << 16)};
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (q < cnt) o[at + q] = h[q];
    }
  };
  if (e.z) put(e.z, a);
  if (e.z_up) put(e.z_up, b);
  if (e.residual) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (q < cnt)
        v[q] += e.f32 ? static_cast<const float*>(e.residual)[at + q]
                      : bf2f(static_cast<const uint16_t*>(e.residual)[at + q]);
  }
  if (!e.f32) {
    put(static_cast<uint16_t*>(e.out), v);
  } else if (vec) {
    *reinterpret_cast<floatx4*>(static_cast<float*>(e.out) + at) = floatx4{v[0], v[1], v[2], v[3]};
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (q < cnt) static_cast<float*>(e.out)[at + q] = v[q];
  }
}

struct Gemm {
  Operand a;          // output rows m
  Operand b0, b1;     // output columns n; b1: the up matrix (DUAL) or the second reduction segment (SEGS = 2)
  int64_t M;
  int N;
  int64_t R;          // reduction length (of one segment)
  int64_t a_seg;      // SEGS = 2: element offset of A's second segment
  Epilogue e;
};

// One BM x BN output tile per workgroup (DUAL: BN columns of both matrices), 4 wavefronts in 2 x 2.
template <int BM, int BN, bool A_COLS, bool B_COLS, bool DUAL, int SEGS>
__global__ __launch_bounds__(256) void gemm_kernel(Gemm g, int mt, int nt) {
  constexpr int NMAT = DUAL ? 2 : 1;
  constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128;
  constexpr int TM = BM / 64, TN = BN / 64;
  __shared__ __attribute__((aligned(1024))) char smem[A_BYTES + NMAT * B_BYTES];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int64_t m0 = (int64_t)(blockIdx.x / nt) * BM;
  const int n0 = (int)(blockIdx.x % nt) * BN;
  floatx16 acc[NMAT][TN][TM];
#pragma unroll
  for (int m = 0; m < NMAT; ++m)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[m][j][i][v] = 0.f;

  // Stage reduction indices [r0, r0 + 64) of operand rows [c0, c0 + C) into `tile`.
  auto stage = [&](auto cols, auto width, const Operand& o, int64_t c0, int64_t r0, char* tile) {
    constexpr bool COLS = decltype(cols)::value;
    constexpr int C = decltype(width)::value;
#pragma unroll
    for (int q = 0; q < C / 32; ++q) {
      const int line = q * 4 + wave;
      uint32_t off = kOut;
      __amdgpu_buffer_rsrc_t rs;
      if (!COLS) {
        const int row = line * 8 + (lane >> 3), chunk = (lane & 7) ^ swz(row);
        const int64_t left = o.rows - c0 < C ? o.rows - c0 : C;
        // (the last chunk of a row may reach past R, into the zeros that pad dz)
        rs = make_rsrc(o.p + c0 * o.ld + r0, ((left - 1) * o.ld + (g.R - r0 + 7) / 8 * 8) * 2);
        if (row < left && r0 + chunk * 8 < g.R) off = (uint32_t)((row * o.ld + chunk * 8) * 2);
      } else {
        constexpr int LPR = C / 8;  // lanes per LDS row
        const int r = line * (64 / LPR) + lane / LPR, chunk = (lane % LPR) ^ swz_t<C>(r);
        const int64_t left = g.R - r0 < BK ? g.R - r0 : BK;
        rs = make_rsrc(o.p + r0 * o.ld + c0, ((left - 1) * o.ld + (o.rows - c0)) * 2);
        if (r < left && c0 + chunk * 8 < o.rows) off = (uint32_t)((r * o.ld + chunk * 8) * 2);
      }
      const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(rs, off, 0, 0);
      *reinterpret_cast<u32x4*>(tile + line * 1024 + lane * 16) = v;
    }
  };
  char* sA = smem;
  char* sB = smem + A_BYTES;
#pragma unroll
  for (int sg = 0; sg < SEGS; ++sg) {
    Operand a = g.a;
    a.p += sg * g.a_seg;
    const Operand b = sg ? g.b1 : g.b0;
    for (int64_t r0 = 0; r0 < g.R; r0 += BK) {
      stage(std::bool_constant<A_COLS>{}, std::integral_constant<int, BM>{}, a, m0, r0, sA);
      stage(std::bool_constant<B_COLS>{}, std::integral_constant<int, BN>{}, b, n0, r0, sB);
      if (DUAL) stage(std::bool_constant<B_COLS>{}, std::integral_constant<int, BN>{}, g.b1, n0, r0, sB + B_BYTES);
      __syncthreads();
#pragma unroll
      for (int ks = 0; ks < BK / 16; ++ks) {
        bf16x8 fa[TM], fb[NMAT][TN];
#pragma unroll
        for (int i = 0; i < TM; ++i) fa[i] = fragment<A_COLS, BM>(sA, wm * (BM / 2) + i * 32, ks, lane);
#pragma unroll
        for (int m = 0; m < NMAT; ++m)
#pragma unroll
          for (int j = 0; j < TN; ++j) fb[m][j] = fragment<B_COLS, BN>(sB + m * B_BYTES, wn * (BN / 2) + j * 32, ks, lane);
#pragma unroll
        for (int m = 0; m < NMAT; ++m)
#pragma unroll
          for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int i = 0; i < TM; ++i)
              acc[m][j][i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fb[m][j], fa[i], acc[m][j][i], 0, 0, 0);
      }
      __syncthreads();
    }
  }
  // The weight side feeds the MFMA's rows, so a lane holds, for output row lane % 32 of each 32-row block,
  // columns 8 q + 4 (lane / 32) + 0..3 (q = 0..3) of each 32-column block.
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int64_t row = m0 + wm * (BM / 2) + i * 32 + (lane & 31);
    if (row >= g.M) continue;
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int n = n0 + wn * (BN / 2) + j * 32 + q * 8 + (lane >> 5) * 4;
        if (n >= g.N) continue;
        float v[4], u[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          v[r] = acc[0][j][i][q * 4 + r];
          u[r] = acc[NMAT - 1][j][i][q * 4 + r];
        }
        store4(g.e, row, n, g.N, v, u);
      }
  }
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

template <int BM, int BN, bool A_COLS, bool B_COLS, bool DUAL, int SEGS>
hipError_t run_gemm(const Gemm& g, hipStream_t s) {
  const int64_t mt = (g.M + BM - 1) / BM, nt = (g.N + BN - 1) / BN;
  if (mt * nt > INT32_MAX) return hipErrorInvalidValue;
  hipLaunchKernelGGL((gemm_kernel<BM, BN, A_COLS, B_COLS, DUAL, SEGS>), dim3((unsigned)(mt * nt)), dim3(256), 0, s, g,
                     (int)mt, (int)nt);
  return hipGetLastError();
}

}  // namespace

size_t linear_ws_bytes(int64_t, int, int, int) { return 0; }

hipError_t launch_linear(const LinearArgs& a, hipStream_t s) {
  Gemm g{};
  g.a = {a.x, a.K, a.M};
  g.b0 = {a.w, a.K, a.N};
  g.b1 = {a.w_up, a.K, a.N};
  g.M = a.M;
  g.N = a.N;
  g.R = a.K;
  g.e = {a.bias, a.bias_up, a.residual, a.out, a.z, a.z_up, a.act, a.out_f32};
  if (a.act == ACT_SWIGLU) return run_gemm<128, 64, false, false, true, 1>(g, s);
  return run_gemm<128, 128, false, false, false, 1>(g, s);
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
    g.a = {dz, ld, a.M};
    g.a_seg = Np;
    g.b0 = {a.w, a.K, a.K};
    g.b1 = {a.w_up, a.K, a.K};
    g.M = a.M;
    g.N = a.K;
    g.R = a.N;
    g.e.out = a.d_x;
    e = mats == 2 ? run_gemm<128, 128, false, true, false, 2>(g, s) : run_gemm<128, 128, false, true, false, 1>(g, s);
    if (e != hipSuccess) return e;
  }
  for (int m = 0; m < mats; ++m) {
    uint16_t* d_w = m ? a.d_w_up : a.d_w;
    if (!d_w) continue;
    g.a = {dz + m * Np, ld, Np};
    g.b0 = {a.x, a.K, a.K};
    g.M = a.N;
    g.N = a.K;
    g.R = a.M;
    g.e.out = d_w;
    e = run_gemm<128, 128, true, true, false, 1>(g, s);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace moe
