// The microscaled formats' elements and scales: a block of 32 consecutive
// numbers shares one power of two (E8M0), the smallest under which no element
// passes the element type's largest value (448 for E4M3, 6 for E2M1), and the
// elements are rounded to nearest, ties to even.
#pragma once
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include <cstdint>

namespace mxfp8 {

// The E8M0 code of a block whose largest magnitude is `top`: 127 for a block
// of zeros; top = f 2^E (1 <= f < 2) takes E - 8 for f <= 1.75, else E - 7.
__device__ __forceinline__ uint32_t scale_code(float top) {
  const uint32_t bits = __float_as_uint(top);
  if (bits == 0u) return 127u;
  const int e = static_cast<int>(bits >> 23) - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return static_cast<uint32_t>(min(max(e, 0), 254));
}
// The same for E2M1: E - 2 for f <= 1.5, else E - 1.
__device__ __forceinline__ uint32_t scale_code_e2m1(float top) {
  const uint32_t bits = __float_as_uint(top);
  if (bits == 0u) return 127u;
  const int e = static_cast<int>(bits >> 23) - 2 + ((bits & 0x7FFFFFu) > 0x400000u ? 1 : 0);
  return static_cast<uint32_t>(min(max(e, 0), 254));
}

// 2^(127 - code), code up to 254 (for which it is subnormal), and 2^(code - 127), NaN for
// the code 255.  An element times the first is exact wherever the element type's codes
// tell values apart.
__device__ __forceinline__ float inverse_scale(uint32_t code) {
  return __uint_as_float(code < 254u ? (254u - code) << 23 : 0x00400000u);
}
__device__ __forceinline__ float scale_of(uint32_t code) {
  return __uint_as_float(code == 0u ? 0x00400000u : code == 255u ? 0x7FC00000u : code << 23);
}

// Two E4M3 codes of v 2^(127 - code).
__device__ __forceinline__ uint32_t to_e4m3(float a, float b, uint32_t code) {
  const float s = inverse_scale(code);
  return __nv_cvt_float2_to_fp8x2(make_float2(a * s, b * s), __NV_SATFINITE, __NV_E4M3);
}
// Two E2M1 codes in a byte, a's in its low half.
__device__ __forceinline__ uint32_t to_e2m1(float a, float b, uint32_t code) {
  const float s = inverse_scale(code);
  return __nv_cvt_float2_to_fp4x2(make_float2(a * s, b * s), __NV_E2M1, cudaRoundNearest);
}

}  // namespace mxfp8
