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

}  // namespace moe
