// 4-bit weights from float32, bf16 or half ones and back (format in weights4.hpp).
#include <algorithm>

#include "kernels.hpp"
#include "rows.hpp"
#include "weights4.hpp"

namespace moe {

namespace {

// One block of 32 weights a thread.
template <typename T>
__global__ void __launch_bounds__(256) weights4_pack_kernel(const T* w, int64_t blocks, uint8_t* codes,
                                                           uint8_t* scales) {
  for (int64_t b = (int64_t)blockIdx.x * 256 + threadIdx.x; b < blocks; b += (int64_t)gridDim.x * 256) {
    float v[kW4Block];
#pragma unroll
    for (int q = 0; q < 4; ++q) load_row<8>(w + b * kW4Block + 8 * q, v + 8 * q);
    uint32_t amax = 0;
#pragma unroll
    for (int j = 0; j < kW4Block; ++j) amax = max(amax, __float_as_uint(v[j]) & 0x7fffffffu);
    const bool finite = amax < 0x7f800000u;
    // exponent field of amax less 2, at least 1
    const int scale = finite ? max((int)(amax >> 23) - 2, 1) : 255;
    uint32_t out[4] = {0, 0, 0, 0};
    if (finite) {
#pragma unroll
      for (int j = 0; j < kW4Block; ++j) {
        const float m = ldexpf(fabsf(v[j]), 127 - scale);  // exact: at most 8, and multiples of 2^-149 2^126
        const float step = m < 2.0f ? 0.5f : m < 4.0f ? 1.0f : 2.0f;
        const float q = fminf(rintf(m / step) * step, 6.0f);
        const uint32_t c = q < 2.0f ? (uint32_t)(2.0f * q) : q < 4.0f ? (uint32_t)q + 2u : (uint32_t)q / 2u + 4u;
        out[j >> 3] |= (c | (__float_as_uint(v[j]) >> 31 << 3)) << (4 * (j & 7));
      }
    }
    *reinterpret_cast<u32x4_t*>(codes + b * (kW4Block / 2)) = u32x4_t{out[0], out[1], out[2], out[3]};
    scales[b] = (uint8_t)scale;
  }
}

template <typename T>
__global__ void __launch_bounds__(256) weights4_unpack_kernel(const uint8_t* codes, const uint8_t* scales,
                                                             int64_t blocks, T* out) {
  for (int64_t b = (int64_t)blockIdx.x * 256 + threadIdx.x; b < 4 * blocks; b += (int64_t)gridDim.x * 256) {
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = weight4(codes, scales, b * 8 + j);
    store_row<8>(out + b * 8, v);
  }
}

unsigned grid_of(int64_t threads) { return (unsigned)std::min<int64_t>((threads + 255) / 256, 1 << 20); }

}  // namespace

hipError_t launch_weights4_pack(int dtype, const void* w, int64_t blocks, void* codes, void* scales, hipStream_t s) {
  return with_rows(dtype, [&](auto* t) {
    typedef std::remove_pointer_t<decltype(t)> T;
    weights4_pack_kernel<T><<<grid_of(blocks), 256, 0, s>>>(static_cast<const T*>(w), blocks,
                                                           static_cast<uint8_t*>(codes), static_cast<uint8_t*>(scales));
    return hipGetLastError();
  });
}

hipError_t launch_weights4_unpack(int dtype, const void* codes, const void* scales, int64_t blocks, void* out,
                                  hipStream_t s) {
  return with_rows(dtype, [&](auto* t) {
    typedef std::remove_pointer_t<decltype(t)> T;
    weights4_unpack_kernel<T><<<grid_of(4 * blocks), 256, 0, s>>>(
        static_cast<const uint8_t*>(codes), static_cast<const uint8_t*>(scales), blocks, static_cast<T*>(out));
    return hipGetLastError();
  });
}

}  // namespace moe
