// Rows of activations in the three storage types (float32, bf16, IEEE half): E
// consecutive elements as float32 and back, one rounding to nearest even each.
#pragma once
#include <type_traits>

#include "common.hpp"

namespace moe {

typedef _Float16 half_t;

// Two float32 values as bf16, rounded to nearest even by gfx950's v_cvt_pk_bf16_f32 (NaN
// stays NaN, subnormals are kept).
__device__ __forceinline__ uint32_t cvt_bf16x2(float lo, float hi) {
  typedef float f32x2_t __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_t{lo, hi}), bf16x2_t));
}

// E elements at p (16-byte aligned rows, E-element aligned columns): 8 of any type, or 4
// float32 ones.
template <int E>
__device__ __forceinline__ void load_row(const float* p, float* v) {
#pragma unroll
  for (int q = 0; q < E / 4; ++q) {
    const f32x4_t a = *reinterpret_cast<const f32x4_t*>(p + 4 * q);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[4 * q + j] = a[j];
  }
}
template <int E>
__device__ __forceinline__ void load_row(const bf16_t* p, float* v) {
  static_assert(E == 8);
  const u32x4_t a = *reinterpret_cast<const u32x4_t*>(p);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = __uint_as_float(a[j] << 16);
    v[2 * j + 1] = __uint_as_float(a[j] & 0xffff0000u);
  }
}
template <int E>
__device__ __forceinline__ void load_row(const half_t* p, float* v) {
  static_assert(E == 8);
  const f16x8_t a = *reinterpret_cast<const f16x8_t*>(p);
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = (float)a[j];
}

template <int E>
__device__ __forceinline__ void store_row(float* p, const float* v) {
#pragma unroll
  for (int q = 0; q < E / 4; ++q)
    *reinterpret_cast<f32x4_t*>(p + 4 * q) = f32x4_t{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
}
template <int E>
__device__ __forceinline__ void store_row(bf16_t* p, const float* v) {
  static_assert(E == 8);
  *reinterpret_cast<u32x4_t*>(p) = u32x4_t{cvt_bf16x2(v[0], v[1]), cvt_bf16x2(v[2], v[3]),
                                           cvt_bf16x2(v[4], v[5]), cvt_bf16x2(v[6], v[7])};
}
template <int E>
__device__ __forceinline__ void store_row(half_t* p, const float* v) {
  static_assert(E == 8);
  *reinterpret_cast<u32x4_t*>(p) = u32x4_t{pack_f16x2(v[0], v[1]), pack_f16x2(v[2], v[3]),
                                           pack_f16x2(v[4], v[5]), pack_f16x2(v[6], v[7])};
}

// E consecutive elements as loaded, converted where they are used: a load whose result
// is converted inside a conditional block would be waited for in that block.
template <typename T, int E>
struct RawRow {
  typedef uint32_t vec_t __attribute__((ext_vector_type(E * sizeof(T) / 4)));
  vec_t v;
  __device__ __forceinline__ void load(const T* p) { v = *reinterpret_cast<const vec_t*>(p); }
  __device__ __forceinline__ void zero() { v = vec_t(0); }
  __device__ __forceinline__ float operator[](int j) const {
    if constexpr (sizeof(T) == 4) {
      return __uint_as_float(v[j]);
    } else {
      const uint32_t w = v[j >> 1];
      if constexpr (std::is_same<T, bf16_t>::value) return __uint_as_float(j & 1 ? w & 0xffff0000u : w << 16);
      return (float)__builtin_bit_cast(f16x2_t, w)[j & 1];
    }
  }
};

// Calls f with a null pointer of the element type that dtype (moe_dtype) names.
template <typename F>
hipError_t with_rows(int dtype, F&& f) {
  switch (dtype) {
    case MOE_F32: return f(static_cast<float*>(nullptr));
    case MOE_BF16: return f(static_cast<bf16_t*>(nullptr));
    case MOE_F16: return f(static_cast<half_t*>(nullptr));
  }
  return hipErrorInvalidValue;
}

}  // namespace moe
