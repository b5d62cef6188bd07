// e4m3 codes with power-of-two block scales: the arithmetic shared by the
// quantising kernels (norm.cu, fp8.cu).
//
// A block's scale is 2^e with the smallest e for which its largest magnitude
// fits into 448 = 1.75 * 2^8 (the largest e4m3 value), stored as the e8m0 byte
// e + 127.  With amax = f * 2^x, 1 <= f < 2: e = x - 8, plus one when f > 1.75;
// read off amax's bits, so no rounding decides it.  Multiplying by 2^-e is
// exact, and nothing saturates.
#pragma once

#include <cuda_fp8.h>

#include "sp24_device.cuh"

namespace sp24 {

constexpr uint32_t kScaleOne = 127u;    // e8m0 byte of 2^0
constexpr uint32_t kScaleNan = 255u;    // e8m0 NaN: the block holds an inf or a NaN

// e8m0 byte of a block from the bit pattern of its largest |value| (bits
// compare like magnitudes, NaNs above infinity).  An empty block has scale 1, a
// block of subnormals 2^-126.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits) {
  // the addend carries into the exponent when the fraction is above 1.75
  const int b = static_cast<int>((amax_bits + 0x1FFFFFu) >> 23) - 8;
  uint32_t byte = static_cast<uint32_t>(max(b, 1));
  byte = amax_bits == 0u ? kScaleOne : byte;
  return amax_bits >= 0x7F800000u ? kScaleNan : byte;
}

// 2^-e of a byte: 2^(127 - byte), or NaN, which makes every code of the block
// NaN (0x7F).
__device__ __forceinline__ float scale_inverse(uint32_t byte) {
  return __uint_as_float(byte == kScaleNan ? 0x7FFFFFFFu : (254u - byte) << 23);
}

// Larger and smaller of two pairs of 16-bit numbers.
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t min_u16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("min.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Four e4m3 codes, a in the low byte: round to nearest even (at most half a
// step, 2^-4 of a normal value).
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

}  // namespace sp24
