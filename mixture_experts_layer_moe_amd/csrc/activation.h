// Device helpers shared by the products' kernels: buffer resources, bf16 widening, MXFP4 scales, activations.
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
