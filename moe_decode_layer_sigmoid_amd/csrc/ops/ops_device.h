// Device helpers of the operators beside the MoE layer.
#pragma once

#include "device_common.h"

namespace moe {

typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));

// e of the least power of two with amax <= 448 * 2^e, at least -127 (amax
// finite and not negative).  448 = 1.75 * 2^8: a mantissa above 1.75 carries
// into the exponent.
__device__ __forceinline__ int scale_exp(float amax) {
  return max(static_cast<int>((__float_as_uint(amax) + 0x1fffffu) >> 23) - 135, -127);
}

// 2^e as a float, e in [-149, 127].
__device__ __forceinline__ float pow2f(int e) {
  return e >= -126 ? __uint_as_float(static_cast<uint32_t>(e + 127) << 23)
                   : __uint_as_float(1u << (e + 149));
}

// |x| for the running maximum: 0 for an infinity or NaN.
__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a <= 3.402823466e38f ? a : 0.f;
}

// Infinities as NaN (an infinity has no code).
__device__ __forceinline__ float inf_to_nan(float x) {
  return fabsf(x) <= 3.402823466e38f ? x : __uint_as_float(0x7fc00000u);
}

// Four floats of magnitude at most 448, or NaN -> four e4m3fn codes (RNE).
__device__ __forceinline__ uint32_t to_fp8x4(float a, float b, float c, float d) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true));
}

}  // namespace moe
