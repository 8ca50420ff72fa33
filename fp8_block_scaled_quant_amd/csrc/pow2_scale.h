// Power-of-two block scales of the feed-forward operators' quantizers: s is the
// smallest power of two with amax <= max * s, max the format's largest value.
//
// amax arrives as the bits of a non-negative fp32, 1.f * 2^x; the format's
// largest value is 1.t * 2^p.  amax <= max * 2^e holds for e = x - p when
// f <= t and for e = x - p + 1 otherwise, so the E8M0 byte e + 127 comes from
// the bits alone, with no rounding.  amax is floored at 2^-100 (a block of
// zeros gets a scale too, and both s and 1 / s stay normal).
#pragma once

#include "device_common.h"

namespace fp8bsq {

constexpr uint32_t kAmaxFloorBits = 27u << 23;   // 2^-100

// kTopExp, kTopMant: exponent and fp32 mantissa field of the format's maximum.
template <int kTopExp, uint32_t kTopMant>
__device__ __forceinline__ uint32_t pow2_scale_byte(uint32_t amax_bits) {
  const uint32_t a = amax_bits > kAmaxFloorBits ? amax_bits : kAmaxFloorBits;
  return (a >> 23) - kTopExp + ((a & 0x7FFFFFu) > kTopMant ? 1u : 0u);
}

__device__ __forceinline__ uint32_t e4m3_scale_byte(uint32_t amax_bits) {   // 448 = 1.75 * 2^8
  return pow2_scale_byte<8, 0x600000u>(amax_bits);
}
__device__ __forceinline__ uint32_t e2m1_scale_byte(uint32_t amax_bits) {   // 6 = 1.5 * 2^2
  return pow2_scale_byte<2, 0x400000u>(amax_bits);
}

// 2^(byte - 127) and its inverse (bytes 1..253).
__device__ __forceinline__ float pow2_scale(uint32_t byte) { return __uint_as_float(byte << 23); }
__device__ __forceinline__ float pow2_inverse(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

}  // namespace fp8bsq
