// 4-bit weights from float32, bf16 or half ones and back (format in weights4.hpp).
#include <algorithm>

#include "kernels.hpp"
#include "rows.hpp"
#include "weights4.hpp"

namespace moe {

namespace {

// Both directions move bytes: 4.25 bits a weight on one side, 16 or 32 on the other. Four lanes
// share a block, eight weights each, so a wavefront's loads and stores are contiguous. 64 x
// 1536 x 2048 bf16: packed in 88 us, unpacked in 94 (5.8 and 5.4 TB/s; a large copy 5.1 to 5.4); in
// turn, each on what the other has just written, 104 and 82 (there and back 186).
// One lane a block and the rounding in float arithmetic took 258 us there and back, four lanes
// with that rounding 134 us there.

// Codes of eight weights in steps of 2^(scale - 127): the hardware's conversion, which rounds
// to the nearest of the grid, ties to the even code, and takes what is larger to 6.
__device__ __forceinline__ uint32_t codes_of(const float* v, uint32_t scale) {
  uint32_t out = 0;
#if defined(__HIP_DEVICE_COMPILE__)
  const float s = __uint_as_float(scale << 23);
  out = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out, v[0], v[1], s, 0);
  out = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out, v[2], v[3], s, 1);
  out = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out, v[4], v[5], s, 2);
  out = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out, v[6], v[7], s, 3);
#else
  (void)v;
  (void)scale;
#endif
  return out;
}

template <typename T>
__global__ void __launch_bounds__(256) weights4_pack_kernel(const T* w, int64_t pieces, uint32_t* codes,
                                                           uint8_t* scales) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < pieces; i += (int64_t)gridDim.x * 256) {
    float v[8];
    load_row<8>(w + i * 8, v);
    uint32_t amax = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) amax = max(amax, __float_as_uint(v[j]) & 0x7fffffffu);
    amax = max(amax, (uint32_t)__builtin_amdgcn_mov_dpp((int)amax, 0xb1, 0xf, 0xf, true));  // lane ^ 1
    amax = max(amax, (uint32_t)__builtin_amdgcn_mov_dpp((int)amax, 0x4e, 0xf, 0xf, true));  // lane ^ 2
    const bool finite = amax < 0x7f800000u;
    // exponent field of amax less 2, at least 1
    const uint32_t scale = finite ? (uint32_t)max((int)(amax >> 23) - 2, 1) : 255u;
    codes[i] = finite ? codes_of(v, scale) : 0u;
    if ((i & 3) == 0) scales[i >> 2] = (uint8_t)scale;
  }
}

template <typename T>
__global__ void __launch_bounds__(256) weights4_unpack_kernel(const uint32_t* codes, const uint8_t* scales,
                                                             int64_t pieces, T* out) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < pieces; i += (int64_t)gridDim.x * 256) {
    const u32x4_t w = __builtin_bit_cast(u32x4_t, weights4_bf16(codes[i], scales[i >> 2]));
    if constexpr (std::is_same<T, bf16_t>::value) {
      *reinterpret_cast<u32x4_t*>(out + i * 8) = w;
    } else {
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(j & 1 ? w[j >> 1] & 0xffff0000u : w[j >> 1] << 16);
      store_row<8>(out + i * 8, v);
    }
  }
}

unsigned grid_of(int64_t threads) { return (unsigned)std::min<int64_t>((threads + 255) / 256, 1 << 20); }

}  // namespace

// blocks < 2^35 (rows * cols < 2^40): pieces and elements in 64 bits.
hipError_t launch_weights4_pack(int dtype, const void* w, int64_t blocks, void* codes, void* scales, hipStream_t s) {
  return with_rows(dtype, [&](auto* t) {
    typedef std::remove_pointer_t<decltype(t)> T;
    weights4_pack_kernel<T><<<grid_of(4 * blocks), 256, 0, s>>>(
        static_cast<const T*>(w), 4 * blocks, static_cast<uint32_t*>(codes), static_cast<uint8_t*>(scales));
    return hipGetLastError();
  });
}

hipError_t launch_weights4_unpack(int dtype, const void* codes, const void* scales, int64_t blocks, void* out,
                                  hipStream_t s) {
  return with_rows(dtype, [&](auto* t) {
    typedef std::remove_pointer_t<decltype(t)> T;
    weights4_unpack_kernel<T><<<grid_of(4 * blocks), 256, 0, s>>>(
        static_cast<const uint32_t*>(codes), static_cast<const uint8_t*>(scales), 4 * blocks, static_cast<T*>(out));
    return hipGetLastError();
  });
}

}  // namespace moe
