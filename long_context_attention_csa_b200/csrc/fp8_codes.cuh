// E4M3 codes with a power-of-two block scale: the scale of a block's largest
// magnitude, and the codes under it.
#pragma once

#include <cuda_fp8.h>
#include <stdint.h>

namespace csa {

// e + 127 of the smallest e >= -127 with amax <= 448 2^e, for a finite amax =
// 1.m 2^x: 448 = 1.75 2^8, so e = x - 8, one more when 1.m > 1.75; amax below
// 448 2^-127 (zero and subnormals included) gives 0.
__device__ __forceinline__ uint32_t scale_byte(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = (int)(b >> 23) - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  return e > 0 ? (uint32_t)e : 0u;
}

// Infinities become NaN, so that the codes say so (the conversion would
// saturate them) and the block's scale does not.
template <int N>
__device__ __forceinline__ void drop_infinities(float* v) {
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (isinf(v[i])) v[i] = __int_as_float(0x7fffffff);
}

// Codes of v 2^-e, rounded to nearest even (the product is exact: the factor is
// a normal power of two); v holds no infinity.  NaN becomes the NaN code.
__device__ __forceinline__ uint32_t codes4(const float* v, uint32_t byte) {
  const float f = __uint_as_float((254u - byte) << 23);   // 2^(127 - byte), byte <= 247
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(v[0] * f, v[1] * f), __NV_SATFINITE,
                                            __NV_E4M3) |
         ((uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(v[2] * f, v[3] * f), __NV_SATFINITE,
                                             __NV_E4M3)
          << 16);
}

}  // namespace csa
