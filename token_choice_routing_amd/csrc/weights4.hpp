// 4-bit weights: blocks of 32 columns, a code of 4 bits a weight (sign, two exponent bits,
// one mantissa bit: +-{0, 0.5, 1, 1.5, 2, 3, 4, 6}), even columns in the low half of a byte,
// and one scale byte e + 127 a block that stands for 2^e (255: the block is NaN). With amax
// the block's largest magnitude e = max(floor(log2 amax) - 2, -126), so amax 2^-e lies in
// [4, 8): the top two magnitudes 4 and 6 are in use and what passes 5 becomes 6.
#pragma once
#include "common.hpp"

namespace moe {

constexpr int kW4Block = 32;

// Eight weights as bf16 (exact) from a dword of codes and the scale byte: the hardware's
// conversion, which multiplies by the power of two that the float's exponent names; 255 << 23
// gives NaN for every code, 0 stands for 2^-127.
__device__ __forceinline__ bf16x8_t weights4_bf16(uint32_t codes, uint32_t scale) {
  bf16x8_t v = {};
#if defined(__HIP_DEVICE_COMPILE__)
  const float s = __uint_as_float(scale << 23);
  const auto a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, s, 0);
  const auto b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, s, 1);
  const auto c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, s, 2);
  const auto d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, s, 3);
  v = bf16x8_t{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
#else
  (void)codes;
  (void)scale;
#endif
  return v;
}

// Scale bytes with which the codes of 4 and 6 pass the largest float.
__device__ __forceinline__ bool weights4_top(uint32_t scale) { return scale - 253u < 2u; }

// The same weights, or an eighth of them: exactly too (multiples of 2^-131), and below 2^127 at
// every scale byte but 255. The bytes below 4 name no eighth: the weights are divided themselves.
__device__ __forceinline__ bf16x8_t weights4_bf16_divided(uint32_t codes, uint32_t scale, bool eighth) {
  const bool low = scale < 4u;
  u32x4_t w = __builtin_bit_cast(u32x4_t, weights4_bf16(codes, eighth && !low && scale != 255u ? scale - 3u : scale));
  const float by = eighth && low ? 0.125f : 1.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float lo = __uint_as_float(w[i] << 16) * by, hi = __uint_as_float(w[i] & 0xffff0000u) * by;
    w[i] = __float_as_uint(lo) >> 16 | (__float_as_uint(hi) & 0xffff0000u);
  }
  return __builtin_bit_cast(bf16x8_t, w);
}

}  // namespace moe
