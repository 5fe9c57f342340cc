// Device helpers shared by the kernels: buffer resources, bf16 widening, MXFP4 scales, lane shifts, activations.
#pragma once

#include "common.h"
#include "operators.h"

namespace moe {

typedef __attribute__((__vector_size__(4 * sizeof(uint32_t)))) uint32_t u32x4;
typedef __attribute__((__vector_size__(2 * sizeof(uint32_t)))) uint32_t u32x2;

__device__ __forceinline__ float bf2f(uint16_t h) { return __builtin_bit_cast(float, (uint32_t)h << 16); }

// The scale of byte s, 2^(s - 127), as the conversions of 4-bit codes (v_cvt_scalef32_*) take it: they read a float's
// exponent alone, so that 0 is 2^-127 here, and 255 makes NaN.
__device__ __forceinline__ float mxfp4_scale(uint32_t s) { return __builtin_bit_cast(float, s << 23); }

// Raw buffer resource over [base, base + bytes): out-of-range reads return zero.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* base, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, 0x00020000);
}

// Data-parallel primitive: lanes of the enabled rows of 16 get `v` of the lane that CTRL names, `old` where there is none.
template <int CTRL, int ROWS = 0xf>
__device__ __forceinline__ int dpp(int old, int v) {
  return __builtin_amdgcn_update_dpp(old, v, CTRL, ROWS, 0xf, false);
}
// Lanes i of each 16 get lane i + N's, the last N zeros.
template <int N>
__device__ __forceinline__ u32x4 shifted(u32x4 v) {
  if constexpr (N == 0) return v;
  u32x4 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = (uint32_t)dpp<0x100 + N>(0, (int)v[i]);  // row_shl:N
  return o;
}

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

}  // namespace moe
