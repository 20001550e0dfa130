// Grouped products for the few rows of a decode step: 16-bit weights, or 4-bit ones
// (weights4.hpp), plain or as silu(W0 a) * (W1 a). What bounds them is the bytes of the chosen
// experts' weights, read once here and straight into registers: an item is one expert's 32
// weight rows (16 of each matrix for gate/up) times up to 64 of its rows, the four wavefronts
// of a workgroup take a quarter of the reduction each and add their sums in LDS in order.
#include <algorithm>

#include "grouped_mm.hpp"
#include "rows.hpp"
#include "weights4.hpp"

namespace moe {

namespace {

constexpr int kFewRows = 64, kChunk = 128;  // rows an item; reduction steps a wavefront takes at a time

// Eight consecutive elements of a as loaded, and as N bf16 parts whose sum they are: 8
// significant bits each (1 part for bf16, 2 for half, 3 for float32; cut off, not rounded, so
// that the largest values stay finite). A value that is not finite is its first part.
template <typename T>
struct Parts;
template <>
struct Parts<bf16_t> {
  static constexpr int N = 1;
  u32x4_t v;
  __device__ __forceinline__ void load(const bf16_t* p) { v = *reinterpret_cast<const u32x4_t*>(p); }
  __device__ __forceinline__ void keep(bool on) { v = on ? v : u32x4_t{0, 0, 0, 0}; }
  __device__ __forceinline__ void split(bf16x8_t (&o)[1]) const { o[0] = __builtin_bit_cast(bf16x8_t, v); }
};
__device__ __forceinline__ uint32_t high_halves(float lo, float hi) {  // two floats cut to bf16
  return __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302);
}
__device__ __forceinline__ float cut_rest(float v) {  // what cutting v to bf16 leaves; 0 if not finite
  const uint32_t u = __float_as_uint(v);
  return (u & 0x7f800000u) == 0x7f800000u ? 0.0f : v - __uint_as_float(u & 0xffff0000u);
}
template <>
struct Parts<half_t> {
  static constexpr int N = 2;
  f16x8_t v;
  __device__ __forceinline__ void load(const half_t* p) { v = *reinterpret_cast<const f16x8_t*>(p); }
  __device__ __forceinline__ void keep(bool on) { v = on ? v : f16x8_t{}; }
  __device__ __forceinline__ void split(bf16x8_t (&o)[2]) const {
    u32x4_t a, b;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float x = (float)v[2 * j], y = (float)v[2 * j + 1];
      a[j] = high_halves(x, y);
      b[j] = high_halves(cut_rest(x), cut_rest(y));
    }
    o[0] = __builtin_bit_cast(bf16x8_t, a);
    o[1] = __builtin_bit_cast(bf16x8_t, b);
  }
};
template <>
struct Parts<float> {
  static constexpr int N = 3;
  f32x4_t v[2];
  __device__ __forceinline__ void load(const float* p) {
    v[0] = *reinterpret_cast<const f32x4_t*>(p);
    v[1] = *reinterpret_cast<const f32x4_t*>(p + 4);
  }
  __device__ __forceinline__ void keep(bool on) {
    v[0] = on ? v[0] : f32x4_t{};
    v[1] = on ? v[1] : f32x4_t{};
  }
  __device__ __forceinline__ void split(bf16x8_t (&o)[3]) const {
    u32x4_t a, b, c;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float x = v[j >> 1][2 * (j & 1)], y = v[j >> 1][2 * (j & 1) + 1];
      const float x1 = cut_rest(x), y1 = cut_rest(y);
      a[j] = high_halves(x, y);
      b[j] = high_halves(x1, y1);
      c[j] = high_halves(cut_rest(x1), cut_rest(y1));
    }
    o[0] = __builtin_bit_cast(bf16x8_t, a);
    o[1] = __builtin_bit_cast(bf16x8_t, b);
    o[2] = __builtin_bit_cast(bf16x8_t, c);
  }
};

// A lane's weights of one chunk: of weight row lane % 16 in the MFMA's layout, four 16 x 32
// steps. 16-bit: step i holds k = 32 i + 8 (lane / 16) .. + 7. 4-bit: lane group j = lane / 16
// owns block j of the chunk (16 bytes, one scale byte), step i its codes 8 i .. 8 i + 7; the
// rows' elements are taken in the same order, so the products meet.
template <typename T, bool W4>
struct Weights;
template <typename T>
struct Weights<T, false> {
  u32x4_t v[4];
  const T* row;
  __device__ __forceinline__ void at(const GroupedMm& g, int, int64_t r) {
    row = static_cast<const T*>(g.w) + r * g.k_dim;
  }
  __device__ __forceinline__ void load(const Weights& base, int c, int j, int K) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int k = c * kChunk + 32 * i + 8 * j;
      v[i] = *reinterpret_cast<const u32x4_t*>(base.row + (k < K ? k : 0));
    }
  }
  __device__ __forceinline__ bf16x8_t step(int i, bool on) const {
    return __builtin_bit_cast(bf16x8_t, on ? v[i] : u32x4_t{0, 0, 0, 0});
  }
};
template <typename T>
struct Weights<T, true> {
  u32x4_t v;
  uint32_t scale;
  const uint8_t *codes, *scales;
  __device__ __forceinline__ void at(const GroupedMm& g, int matrix, int64_t r) {
    codes = (matrix ? g.codes1 : g.codes0) + r * (g.k_dim / 2);
    scales = (matrix ? g.scales1 : g.scales0) + r * (g.k_dim / kW4Block);
  }
  __device__ __forceinline__ void load(const Weights& base, int c, int j, int K) {
    const int b = c * (kChunk / kW4Block) + j < K / kW4Block ? c * (kChunk / kW4Block) + j : 0;
    v = *reinterpret_cast<const u32x4_t*>(base.codes + b * (kW4Block / 2));
    scale = base.scales[b];
  }
  __device__ __forceinline__ bf16x8_t step(int i, bool on) const {
    return weights4_bf16(on ? v[i] : 0u, on ? scale : 127u);
  }
};

template <typename T, bool W4>
__device__ __forceinline__ f32x4_t mfma_few(bf16x8_t w, bf16x8_t a, f32x4_t c) {
  if constexpr (std::is_same<T, half_t>::value && !W4)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, w), __builtin_bit_cast(f16x8_t, a), c, 0,
                                                  0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, a, c, 0, 0, 0);
}

template <typename T, bool W4, bool SWIGLU>
__global__ void __launch_bounds__(256) grouped_mm_few_kernel(GroupedMm g) {
  constexpr int U = W4 ? (sizeof(T) == 4 ? 2 : 4) : 2;  // chunks in flight
  constexpr int NP = W4 ? Parts<T>::N : 1;
  __shared__ Segments sg;
  __shared__ f32x4_t red[4][kFewRows / 16 * 2][kWave];
  constexpr int OC = SWIGLU ? 16 : 32;  // output columns an item
  const int nt = (g.n_out + OC - 1) / OC;
  const int total = build_segments(sg, g.offsets, g.groups, g.rows, kFewRows, nt, 0);
  const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int l16 = lane & 15, j = lane >> 4;
  const int K = g.k_dim, chunks = (K + kChunk - 1) / kChunk;
  const int c0 = chunks * wave / 4, c1 = chunks * (wave + 1) / 4;
  for (int it = blockIdx.x; it < total; it += gridDim.x) {
    const int e = segment_of(sg, g.groups, it);
    const int mt = (sg.len[e] + kFewRows - 1) / kFewRows, local = it - sg.prefix[e];
    const int n0 = local / mt * OC, r0 = sg.start[e] + local % mt * kFewRows;
    const int rows = __builtin_amdgcn_readfirstlane(min(kFewRows, sg.start[e] + sg.len[e] - r0));
    Weights<T, W4> base[2];
#pragma unroll
    for (int b = 0; b < 2; ++b)
      base[b].at(g, SWIGLU ? b : 0, (int64_t)e * g.n_out + min(n0 + (SWIGLU ? 0 : 16 * b) + l16, g.n_out - 1));
    auto item = [&](auto tiles) __attribute__((always_inline)) {
      constexpr int MT = decltype(tiles)::value;
      f32x4_t acc[MT][2];
      const T* arow[MT];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        acc[m][0] = acc[m][1] = f32x4_t{0, 0, 0, 0};
        int64_t row = r0 + min(16 * m + l16, rows - 1);
        if (g.a_rows) row = min<int64_t>(max<int64_t>(g.a_rows[row], 0), g.a_nrows - 1);
        arow[m] = static_cast<const T*>(g.a) + row * g.lda;
      }
      for (int c = c0; c < c1; c += U) {
        Weights<T, W4> w[U][2];
        Parts<T> a[MT == 1 ? U : 1][4];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int cu = min(c + u, c1 - 1);
#pragma unroll
          for (int b = 0; b < 2; ++b) w[u][b].load(base[b], cu, j, K);
        }
        // element order of a chunk's step i: as the weights'
        auto col = [&](int cu, int i) { return cu * kChunk + (W4 ? 32 * j + 8 * i : 32 * i + 8 * j); };
        auto load = [&](Parts<T>(&x)[4], const T* p, int cu) __attribute__((always_inline)) {
#pragma unroll
          for (int i = 0; i < 4; ++i) x[i].load(p + (col(cu, i) < K ? col(cu, i) : 0));
        };
        if (MT == 1) {
#pragma unroll
          for (int u = 0; u < U; ++u) load(a[u], arow[0], min(c + u, c1 - 1));
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int cu = c + u;
          if (cu >= c1) break;
          bf16x8_t wf[4][2];
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int b = 0; b < 2; ++b) wf[i][b] = w[u][b].step(i, col(cu, i) < K);
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            if (MT > 1 && 16 * m >= rows) break;
            Parts<T>(&x)[4] = a[MT == 1 ? u : 0];
            if (MT > 1) load(x, arow[m], cu);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              x[i].keep(col(cu, i) < K);
              bf16x8_t p[NP];
              if constexpr (W4) x[i].split(p);
              else p[0] = __builtin_bit_cast(bf16x8_t, x[i].v);
#pragma unroll
              for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int q = 0; q < NP; ++q) acc[m][b] = mfma_few<T, W4>(wf[i][b], p[NP - 1 - q], acc[m][b]);
            }
          }
        }
      }
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int b = 0; b < 2; ++b) red[wave][2 * m + b][lane] = acc[m][b];
      __syncthreads();
      // lane: row l16 of 16, four columns 4 j .. of 16
      auto sum = [&](int q) __attribute__((always_inline)) {
        return (red[0][q][lane] + red[1][q][lane]) + (red[2][q][lane] + red[3][q][lane]);
      };
#pragma unroll
      for (int q = 0; q < (SWIGLU ? MT : 2 * MT); ++q) {
        if ((q & 3) != wave) continue;
        const int r = 16 * (SWIGLU ? q : q / 2) + l16, n = n0 + (SWIGLU ? 0 : 16 * (q & 1)) + 4 * j;
        f32x4_t v = sum(SWIGLU ? 2 * q : q);
        if constexpr (SWIGLU) {
          const f32x4_t up = sum(2 * q + 1);
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = silu(v[i]) * up[i];
        }
        if (r >= rows || n >= g.n_out) continue;
        const int64_t at = (int64_t)(r0 + r) * g.ldo + n;
        if (g.out_dtype == MOE_F32)
          *reinterpret_cast<f32x4_t*>(static_cast<float*>(g.out) + at) = v;
        else if (g.out_dtype == MOE_BF16)
          *reinterpret_cast<u32x2_t*>(static_cast<uint16_t*>(g.out) + at) =
              u32x2_t{cvt_bf16x2(v[0], v[1]), cvt_bf16x2(v[2], v[3])};
        else
          *reinterpret_cast<u32x2_t*>(static_cast<uint16_t*>(g.out) + at) =
              u32x2_t{pack_f16x2(v[0], v[1]), pack_f16x2(v[2], v[3])};
      }
      __syncthreads();  // before the next item's sums
    };
    if (rows <= 16) item(std::integral_constant<int, 1>{});
    else item(std::integral_constant<int, kFewRows / 16>{});
  }
}

}  // namespace

hipError_t launch_grouped_mm_few(const GroupedMm& g, int num_cus, hipStream_t s) {
  const bool w4 = g.form != kMm, swiglu = g.form == kMm4Swiglu;
  const int64_t nt = (g.n_out + (swiglu ? 15 : 31)) / (swiglu ? 16 : 32);
  const int64_t items = (g.rows / kFewRows + std::min<int64_t>(g.groups, g.rows)) * nt;
  const unsigned blocks = (unsigned)std::min<int64_t>(items, 4 * num_cus);
  return with_rows(g.dtype, [&](auto* t) {
    typedef std::remove_pointer_t<decltype(t)> T;
    if (!w4) {
      if constexpr (sizeof(T) == 2) grouped_mm_few_kernel<T, false, false><<<blocks, 256, 0, s>>>(g);
      else return hipErrorInvalidValue;
    } else if (swiglu) {
      grouped_mm_few_kernel<T, true, true><<<blocks, 256, 0, s>>>(g);
    } else {
      grouped_mm_few_kernel<T, true, false><<<blocks, 256, 0, s>>>(g);
    }
    return hipGetLastError();
  });
}

}  // namespace moe
