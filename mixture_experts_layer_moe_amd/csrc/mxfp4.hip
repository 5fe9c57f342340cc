// MXFP4 (OCP microscaling format): values in 4 bits with a shared scale per 32.
//
//   block  32 consecutive values along the last dimension
//   scale  one byte s: 2^(s - 127); 255 makes the whole block NaN
//   code   e2m1, sign and {0, .5, 1, 1.5, 2, 3, 4, 6}; the even value in the low half of a byte
//
// Quantising takes s - 127 = floor(log2 max|x|) - 2, so that the largest value lies in [4, 8) grid units, and rounds
// x / 2^(s - 127) to the nearest grid value, ties to even, saturated at 6 (the format's own rule: the largest values of
// a block lose up to a quarter, all others half a grid step).  The rows follow one another without a gap and are whole
// blocks, so both directions run over a flat sequence of blocks.
//
// A block is four lanes of eight values: 16 bytes a lane of bf16 (32 of fp32), 4 bytes of codes, so that loads and
// stores of a wavefront are contiguous; the maximum goes round the quad by DPP.  The conversions are the hardware's
// (v_cvt_scalef32_*), which take the scale as the exponent of a float.
#include "activation.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kUnits = 4;  // lane units of eight values a thread has in flight

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

// Eight values as fp32.
template <bool F32>
struct Eight {
  u32x4 r[F32 ? 2 : 1];
  __device__ __forceinline__ float operator[](int i) const {
    if (F32) return __builtin_bit_cast(float, (uint32_t)r[i >> 2][i & 3]);
    return bf2f((uint16_t)(r[0][i >> 1] >> (16 * (i & 1))));
  }
};

// HBM-bound: 90112 x 2048 in bf16 109 us (467 MB, 4.3 TB/s), back 69 us; 64 x 7168 2.8 and 2.5 us, a launch.
template <bool F32>
__global__ __launch_bounds__(kThreads) void quantize_kernel(const u32x4* __restrict__ x, int64_t units,
                                                            uint32_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  const int64_t u0 = (int64_t)blockIdx.x * (kThreads * kUnits) + threadIdx.x;
  Eight<F32> v[kUnits];
#pragma unroll
  for (int q = 0; q < kUnits; ++q) {
    const int64_t u = u0 + q * kThreads;
    if (u < units) {
#pragma unroll
      for (int p = 0; p < (F32 ? 2 : 1); ++p) v[q].r[p] = x[u * (F32 ? 2 : 1) + p];
    }
  }
#pragma unroll
  for (int q = 0; q < kUnits; ++q) {
    const int64_t u = u0 + q * kThreads;
    if (u >= units) return;  // (a block's four units exist together, so a quad's lanes leave together)
    // Magnitudes order as their bits do, infinities and NaN above all numbers.
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float f = v[q][i];
      const uint32_t m = __builtin_bit_cast(uint32_t, f) & 0x7fffffffu;
      top = m > top ? m : top;
    }
    uint32_t o = (uint32_t)dpp<0xB1>(0, (int)top);  // quad_perm [1,0,3,2]
    top = o > top ? o : top;
    o = (uint32_t)dpp<0x4E>(0, (int)top);           // quad_perm [2,3,0,1]
    top = o > top ? o : top;
    const uint32_t e = top >> 23, s = e == 255 ? 255 : e > 2 ? e - 2 : 0;
    const float scale = mxfp4_scale(s);
    uint32_t c = 0;
    if (e != 255) {
      c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[q][0], v[q][1], scale, 0);
      c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[q][2], v[q][3], scale, 1);
      c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[q][4], v[q][5], scale, 2);
      c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[q][6], v[q][7], scale, 3);
    }
    codes[u] = c;
    if ((threadIdx.x & 3) == 0) scales[u >> 2] = (uint8_t)s;
  }
}

// A lane stores 16 bytes, side by side with its neighbours': eight values in bf16, four in fp32 (eight, as two stores of
// 16 bytes in each 32, 11.0 us instead of 8.1 at 5003 x 1440).
template <bool F32>
__global__ __launch_bounds__(kThreads) void dequantize_kernel(const void* __restrict__ codes, const uint8_t* __restrict__ scales,
                                                              int64_t units, u32x4* __restrict__ out) {
  const int64_t u0 = (int64_t)blockIdx.x * (kThreads * kUnits) + threadIdx.x;
  uint32_t c[kUnits], s[kUnits];
#pragma unroll
  for (int q = 0; q < kUnits; ++q) {
    const int64_t u = u0 + q * kThreads;
    if constexpr (F32) c[q] = u < units ? static_cast<const uint16_t*>(codes)[u] : 0;
    else c[q] = u < units ? static_cast<const uint32_t*>(codes)[u] : 0;
    s[q] = u < units ? scales[u >> (F32 ? 3 : 2)] : 0;
  }
#pragma unroll
  for (int q = 0; q < kUnits; ++q) {
    const int64_t u = u0 + q * kThreads;
    if (u >= units) return;
    const float scale = mxfp4_scale(s[q]);
    if constexpr (F32) {
      const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[q], scale, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[q], scale, 1);
      out[u] = __builtin_bit_cast(u32x4, floatx4{a.x, a.y, b.x, b.y});
    } else {
      // (every value has two significant bits: exact in bf16, subnormal ones included)
      const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[q], scale, 0), b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[q], scale, 1);
      const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[q], scale, 2), e = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[q], scale, 3);
      out[u] = u32x4{__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b), __builtin_bit_cast(uint32_t, d),
                     __builtin_bit_cast(uint32_t, e)};
    }
  }
}

}  // namespace

hipError_t launch_mxfp4_quantize(const void* x, bool f32, int64_t blocks, uint8_t* codes, uint8_t* scales, hipStream_t s) {
  const int64_t units = blocks * 4;
  const dim3 grid((unsigned)((units + kThreads * kUnits - 1) / (kThreads * kUnits)));
  const u32x4* src = static_cast<const u32x4*>(x);
  uint32_t* dst = reinterpret_cast<uint32_t*>(codes);
  if (f32) hipLaunchKernelGGL(quantize_kernel<true>, grid, dim3(kThreads), 0, s, src, units, dst, scales);
  else hipLaunchKernelGGL(quantize_kernel<false>, grid, dim3(kThreads), 0, s, src, units, dst, scales);
  return hipGetLastError();
}

hipError_t launch_mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t blocks, bool f32, void* out,
                                   hipStream_t s) {
  const int64_t units = blocks * (f32 ? 8 : 4);
  const int64_t groups = (units + kThreads * kUnits - 1) / (kThreads * kUnits);
  if (groups * kThreads > UINT32_MAX) return hipErrorNotSupported;  // (a grid holds fewer than 2^32 threads)
  const dim3 grid((unsigned)groups);
  u32x4* dst = static_cast<u32x4*>(out);
  if (f32) hipLaunchKernelGGL(dequantize_kernel<true>, grid, dim3(kThreads), 0, s, codes, scales, units, dst);
  else hipLaunchKernelGGL(dequantize_kernel<false>, grid, dim3(kThreads), 0, s, codes, scales, units, dst);
  return hipGetLastError();
}

}  // namespace moe
