// kvq.cuh -- the 8-bit cache's number formats: e4m3 codes and power-of-two
// scales held as biased exponents (e8m0).
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"

namespace simsd {

constexpr int kExpLo = -64, kExpHi = 7;   // range of a page's scale exponent
constexpr int kScaleBias = 127;
constexpr int kScaleNan = 255;            // e8m0 NaN: a page that got a NaN or an infinity

// 2^e for -126 <= e <= 127.
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// Value of a stored scale byte: 2^(byte - 127), NaN for 255.  (0 stands for
// 2^-127; the append writes 63..134 and 255.)
__device__ __forceinline__ float scale_value(uint32_t byte) {
  return byte == kScaleNan ? __uint_as_float(0x7fc00000u)
         : byte == 0 ? __uint_as_float(0x00400000u) : __uint_as_float(byte << 23);
}

// Smallest exponent E in lo..hi with amax <= 448 * 2^E (448 = 1.75 * 2^8, so
// the mantissa decides between exponent - 8 and one more); amax past the
// range takes hi.  The caller handles NaN and infinity.
__device__ __forceinline__ int scale_exponent(float amax, int lo = kExpLo, int hi = kExpHi) {
  const uint32_t u = __float_as_uint(amax);
  const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return min(max(e, lo), hi);
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// Two fp32 values to e4m3 codes (round to nearest even, saturating), lo in
// the low byte.
__device__ __forceinline__ uint32_t pack_e4m3x2(float lo, float hi) {
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

// Two e4m3 codes (low 16 bits) to fp32: exact through fp16.
__device__ __forceinline__ float2 unpack_e4m3x2(uint32_t codes) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)codes, __NV_E4M3);
  return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

}  // namespace simsd
