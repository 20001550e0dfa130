// 4-bit weights: blocks of 32 columns, a code of 4 bits a weight (sign, two exponent bits,
// one mantissa bit: +-{0, 0.5, 1, 1.5, 2, 3, 4, 6}), even columns in the low half of a byte,
// and one scale byte e + 127 a block that stands for 2^e (255: the block is NaN). With amax
// the block's largest magnitude e = max(floor(log2 amax) - 2, -126), so amax 2^-e lies in
// [4, 8): the top two magnitudes 4 and 6 are in use and what passes 5 becomes 6.
#pragma once
#include "common.hpp"

namespace moe {

constexpr int kW4Block = 32;

// The weight at flat element i of a matrix whose rows are whole blocks.
__device__ __forceinline__ float weight4(const uint8_t* codes, const uint8_t* scales, int64_t i) {
  const uint32_t q = codes[i >> 1] >> (4 * (i & 1)) & 15u, s = scales[i / kW4Block];
  const uint32_t m = q & 7u;
  const float v = m < 2 ? 0.5f * (float)m : (float)(2 + (m & 1)) * (float)(1 << (m >> 1)) * 0.25f;
  const float w = s == 255u ? __uint_as_float(0x7fc00000u) : ldexpf(v, (int)s - 127);
  return q & 8u ? -w : w;
}

}  // namespace moe
