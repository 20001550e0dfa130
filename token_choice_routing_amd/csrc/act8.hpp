// Encoding of the 8-bit activation checkpoints (blocks of 32 columns, int8 codes and a
// power-of-two scale byte; act8.hip has the format).
#pragma once
#include "common.hpp"

namespace moe {

// Magnitudes as integers order like the floats, with NaN above infinity.
__device__ __forceinline__ uint32_t act8_magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// Scale byte of a block from its largest magnitude: the biased exponent of amax less 6,
// at least 1 (below 2^-120); 255 for a NaN or an infinity.
__device__ __forceinline__ uint32_t act8_scale(uint32_t amax) {
  const int m = (int)(amax >> 23);
  return m == 255 ? 255u : (uint32_t)max(m - 6, 1);
}

// Four codes: v 2^-e + 1.5 2^23 rounds to an integer (nearest even) in the low bits.
__device__ __forceinline__ uint32_t act8_encode(float v0, float v1, float v2, float v3, uint32_t scale) {
  if (scale == 255) return 0;
  const float inv = __uint_as_float((254 - scale) << 23);  // 2^-e
  constexpr float kMagic = 12582912.0f;
  auto code = [&](float v) {
    return __float_as_uint(fminf(fmaxf(fmaf(v, inv, kMagic), kMagic - 127.0f), kMagic + 127.0f)) & 0xff;
  };
  return code(v0) | (code(v1) << 8) | (code(v2) << 16) | (code(v3) << 24);
}

}  // namespace moe
