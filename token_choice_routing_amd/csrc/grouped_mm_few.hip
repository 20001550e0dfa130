// Grouped products for the few rows of a decode step: 16-bit weights, or 4-bit ones
// (weights4.hpp), plain or as silu(W0 a) * (W1 a). What bounds them is the bytes of the chosen
// experts' weights, read once here and straight into registers: an item is one expert's 32
// weight rows (16 of each matrix for gate/up) times up to 16 or 64 of its rows. It belongs to one
// wavefront, or to the four of a workgroup, which take a quarter of the reduction each and add
// their sums in LDS in order.
#include <algorithm>

#include "grouped_mm.hpp"
#include "rows.hpp"
#include "weights4.hpp"

namespace moe {

namespace {

constexpr int kChunk = 128;  // elements of the reduction that a wavefront takes at a time

// Eight consecutive elements of a as loaded, and as N bf16 parts whose sum they are: 8
// significant bits each (1 part for bf16, 2 for half, 3 for float32; cut off, not rounded, so
// that the largest values stay finite). A value that is not finite is its first part. Bits below
// bf16's smallest subnormal, 2^-133, are in no part (a float32 of less than 2^-110 may have some).
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
      // (a NaN whose payload is in the bits cut off would become an infinity: quiet it first)
      const float x = __builtin_canonicalizef(v[j >> 1][2 * (j & 1)]);
      const float y = __builtin_canonicalizef(v[j >> 1][2 * (j & 1) + 1]);
      const float x1 = cut_rest(x), y1 = cut_rest(y);
      a[j] = high_halves(x, y);
      b[j] = high_halves(x1, y1);
      c[j] = high_halves(cut_rest(x1), cut_rest(y1));
    }
    o[0] = __builtin_bit_cast(bf16x8_t, a);
    o[1] = __builtin_bit_cast(bf16x8_t, b);
    o[2] = __builtin_bit_cast(bf16x8_t, c);
  }
  // What the parts leave out, times 2^64: 16 bits in two parts.
  __device__ __forceinline__ void left_out(bf16x8_t (&o)[2]) const {
    u32x4_t a, b;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float r[2];
#pragma unroll
      for (int h = 0; h < 2; ++h)
        r[h] = cut_rest(cut_rest(cut_rest(__builtin_canonicalizef(v[j >> 1][2 * (j & 1) + h])))) * 0x1p64f;
      a[j] = high_halves(r[0], r[1]);
      b[j] = high_halves(cut_rest(r[0]), cut_rest(r[1]));
    }
    o[0] = __builtin_bit_cast(bf16x8_t, a);
    o[1] = __builtin_bit_cast(bf16x8_t, b);
  }
  // m: the smallest magnitude but 0 so far, as bits without the sign less 1 (0 becomes the largest)
  static constexpr uint32_t kWhole = ((127u - 110u) << 24) - 1u;  // 2^-110: from there on nothing is left out
  __device__ __forceinline__ void smallest(uint32_t& m) const {
#pragma unroll
    for (int j = 0; j < 8; j += 2)
      m = min(min((__float_as_uint(v[j >> 2][j & 3]) << 1) - 1u, (__float_as_uint(v[j >> 2][(j & 3) + 1]) << 1) - 1u), m);
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
  // The eight weights from column k on (0 unless on), an eighth of them if asked for.
  __device__ __forceinline__ bf16x8_t one(int k, bool on, bool eighth) const {
    const uint32_t c = on ? *reinterpret_cast<const uint32_t*>(codes + k / 2) : 0u;
    return weights4_bf16_divided(c, on ? scales[k / kW4Block] : 127u, eighth);
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

// KS wavefronts of the workgroup's four share an item's reduction; 4 / KS items run side by
// side, of neighbouring columns. (Two wavefronts a SIMD are named for the items of 64 float32 rows:
// the compiler then puts no sums into accumulation registers, with which it ends at one. 64
// experts of 32 gathered float32 rows, 2048 x 1536: 211 us without, 166 so.)
template <typename T, bool W4, bool SWIGLU, int KS, int MT>
__global__ void __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2))) grouped_mm_few_kernel(GroupedMm g) {
  constexpr int kRows = 16 * MT;
  // of more than 16 rows two sixteens in turn (64 experts of 32 rows: 96 -> 69 us in bf16; float32
  // ones would take too many registers: 131 -> 157)
  constexpr int NA = MT == 1 || sizeof(T) == 4 ? 1 : 2;
  constexpr int NP = W4 ? Parts<T>::N : 1;
  constexpr int OC = SWIGLU ? 16 : 32, WC = OC * (4 / KS);  // output columns of an item, of the workgroup
  __shared__ Segments sg;
  __shared__ f32x4_t red[KS > 1 ? 4 : 1][KS > 1 ? MT * 2 : 1][kWave];
  const int nt = (g.n_out + WC - 1) / WC;
  const int total = build_segments(sg, g.offsets, g.groups, g.rows, kRows, nt, 0);
  const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int l16 = lane & 15, j = lane >> 4;
  const int ks = wave % KS, K = g.k_dim, chunks = (K + kChunk - 1) / kChunk;
  const int c0 = chunks * ks / KS, c1 = chunks * (ks + 1) / KS;
  for (int it = blockIdx.x; it < total; it += gridDim.x) {
    const int e = segment_of(sg, g.groups, it);
    const int mt = (sg.len[e] + kRows - 1) / kRows, local = it - sg.prefix[e];
    const int n0 = local / mt * WC + wave / KS * OC, r0 = sg.start[e] + local % mt * kRows;
    const int rows = __builtin_amdgcn_readfirstlane(min(kRows, sg.start[e] + sg.len[e] - r0));
    auto weights_at = [&](Weights<T, W4> (&w)[2], int l) __attribute__((always_inline)) {
#pragma unroll
      for (int b = 0; b < 2; ++b)
        w[b].at(g, SWIGLU ? b : 0, (int64_t)e * g.n_out + min(n0 + (SWIGLU ? 0 : 16 * b) + l, g.n_out - 1));
    };
    Weights<T, W4> base[2];
    weights_at(base, l16);
    {
      f32x4_t acc[MT][2];
      const T* arow[MT];
#pragma unroll
      for (int m = 0; m < MT; ++m) acc[m][0] = acc[m][1] = f32x4_t{0, 0, 0, 0};
      auto row_at = [&](int r) __attribute__((always_inline)) {
        int64_t row = r0 + min(r, rows - 1);
        if (g.a_rows) row = min<int64_t>(max<int64_t>(g.a_rows[row], 0), g.a_nrows - 1);
        return static_cast<const T*>(g.a) + row * g.lda;
      };
      // the element that a lane's step i of chunk c begins at, in the weights' order
      auto col = [&](int c, int i) { return c * kChunk + (W4 ? 32 * j + 8 * i : 32 * i + 8 * j); };
      struct Set {  // a chunk in registers; two in turn
        Weights<T, W4> w[2];
        Parts<T> a[NA][4];
      };
      auto load_rows = [&](Set& s, int m, int c) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) s.a[m % NA][i].load(arow[m] + (col(c, i) < K ? col(c, i) : 0));
      };
      auto load = [&](Set& s, int c) __attribute__((always_inline)) {
        if (c >= c1) return;
#pragma unroll
        for (int b = 0; b < 2; ++b) s.w[b].load(base[b], c, j, K);
        load_rows(s, 0, c);
      };
      Set s0, s1;
      // lanes (weight row l16) that met a block whose weights may pass the largest float
      uint64_t top[2] = {0, 0};
      uint32_t least = ~0u;  // Parts<float>::smallest() of the lane's rows
      auto multiply = [&](Set& s, int c) __attribute__((always_inline)) {
        if (c >= c1) return;
        if constexpr (W4) {
#pragma unroll
          for (int b = 0; b < 2; ++b) top[b] |= ballot(weights4_top(s.w[b].scale));
        }
        bf16x8_t wf[4][2];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int b = 0; b < 2; ++b) wf[i][b] = s.w[b].step(i, col(c, i) < K);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          if (MT > 1 && 16 * m >= rows) break;
          if (NA == 1 && m > 0) load_rows(s, m, c);
          if (NA == 2 && m + 1 < MT && 16 * (m + 1) < rows) load_rows(s, m + 1, c);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            s.a[m % NA][i].keep(col(c, i) < K);
            if constexpr (W4 && sizeof(T) == 4) s.a[m % NA][i].smallest(least);
            bf16x8_t p[NP];
            if constexpr (W4) s.a[m % NA][i].split(p);
            else p[0] = __builtin_bit_cast(bf16x8_t, s.a[m % NA][i].v);
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
              for (int q = 0; q < NP; ++q) acc[m][b] = mfma_few<T, W4>(wf[i][b], p[NP - 1 - q], acc[m][b]);
          }
        }
      };
      // (the weights of the first chunk are on their way before the rows' numbers are read)
#pragma unroll
      for (int b = 0; b < 2; ++b)
        if (c0 < c1) s0.w[b].load(base[b], c0, j, K);
#pragma unroll
      for (int m = 0; m < MT; ++m) arow[m] = row_at(16 * m + l16);
      if (c0 < c1) load_rows(s0, 0, c0);
      load(s1, c0 + 1);
      for (int c = c0; c < c1; c += 2) {
        multiply(s0, c);
        load(s0, c + 2);
        multiply(s1, c + 1);
        load(s1, c + 3);
      }
      // The wavefront's sums once more, where such a block was met or a row has bits too small for
      // bf16. Weights of 2^128 and more were infinities above, which make NaN of a row's parts that
      // are 0 and infinities of products that are not: the weight rows that hold one are taken
      // divided by 8, and their sums times 8. The bits left out above have sums of their own, times
      // 2^64. (Apart from the loop above, which keeps its registers, the pointers' too: both are
      // hardly ever met.)
      if constexpr (W4) {
        bool small_rows = false;
        if constexpr (sizeof(T) == 4) small_rows = ballot(least < Parts<T>::kWhole) != 0;
        if (__builtin_expect((top[0] | top[1]) != 0 || small_rows, 0)) {
          const int l16 = opaque_v((int)threadIdx.x) & 15;
          Weights<T, W4> base[2];
          weights_at(base, l16);
          uint32_t eighths[2];
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            const uint64_t at = top[b] | top[b] >> 32;
            eighths[b] = (uint32_t)(at | at >> 16) & 0xffffu;
          }
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            if (MT > 1 && 16 * m >= rows) break;
            const T* const row = row_at(16 * m + l16);
            f32x4_t sum[2] = {}, small[2] = {};
#pragma unroll 1
            for (int t = 4 * c0; t < 4 * c1; ++t) {
              const int k = col(t >> 2, t & 3);
              const bool on = k < K;
              Parts<T> a;
              a.load(row + (on ? k : 0));
              a.keep(on);
              bf16x8_t p[NP], r[2];
              a.split(p);
              if constexpr (sizeof(T) == 4) a.left_out(r);
#pragma unroll
              for (int b = 0; b < 2; ++b) {
                const bf16x8_t w = base[b].one(on ? k : 0, on, eighths[b] >> l16 & 1);
#pragma unroll
                for (int q = 0; q < NP; ++q) sum[b] = mfma_few<T, W4>(w, p[NP - 1 - q], sum[b]);
                if constexpr (sizeof(T) == 4) {
                  small[b] = mfma_few<T, W4>(w, r[1], small[b]);
                  small[b] = mfma_few<T, W4>(w, r[0], small[b]);
                }
              }
            }
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
              for (int q = 0; q < 4; ++q)
                acc[m][b][q] = (sum[b][q] + small[b][q] * 0x1p-64f) * (eighths[b] >> (4 * j + q) & 1 ? 8.0f : 1.0f);
          }
        }
      }
      // lane: row l16 of 16, four columns 4 j .. of 16
      auto store = [&](int r, int n, const f32x4_t& v) __attribute__((always_inline)) {
        if (r >= rows || n >= g.n_out) return;
        const int64_t at = (int64_t)(r0 + r) * g.ldo + n;
        if (g.out_dtype == MOE_F32)
          *reinterpret_cast<f32x4_t*>(static_cast<float*>(g.out) + at) = v;
        else if (g.out_dtype == MOE_BF16)
          *reinterpret_cast<u32x2_t*>(static_cast<uint16_t*>(g.out) + at) =
              u32x2_t{cvt_bf16x2(v[0], v[1]), cvt_bf16x2(v[2], v[3])};
        else
          *reinterpret_cast<u32x2_t*>(static_cast<uint16_t*>(g.out) + at) =
              u32x2_t{pack_f16x2(v[0], v[1]), pack_f16x2(v[2], v[3])};
      };
      auto act = [&](f32x4_t v, const f32x4_t& up) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = silu(v[i]) * up[i];
        return v;
      };
      if constexpr (KS == 1) {
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const int r = 16 * m + l16, n = n0 + 4 * j;
          if constexpr (SWIGLU) {
            store(r, n, act(acc[m][0], acc[m][1]));
          } else {
            store(r, n, acc[m][0]);
            store(r, n + 16, acc[m][1]);
          }
        }
      } else {
        static_assert(KS == 4, "the sums below are of four wavefronts");
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int b = 0; b < 2; ++b) red[wave][2 * m + b][lane] = acc[m][b];
        __syncthreads();
        auto sum = [&](int q) __attribute__((always_inline)) {
          return (red[0][q][lane] + red[1][q][lane]) + (red[2][q][lane] + red[3][q][lane]);
        };
#pragma unroll
        for (int q = 0; q < (SWIGLU ? MT : 2 * MT); ++q) {
          if ((q & 3) != wave) continue;
          if constexpr (SWIGLU) store(16 * q + l16, n0 + 4 * j, act(sum(2 * q), sum(2 * q + 1)));
          else store(16 * (q / 2) + l16, n0 + 16 * (q & 1) + 4 * j, sum(q));
        }
        __syncthreads();  // before the next item's sums
      }
    }
  }
}

}  // namespace

// Rules (us at 64 experts, n 2048, k 1536, bf16): a wavefront takes the whole reduction where
// there are items for most of them (64 rows: 33 against 40 with a quarter each; 2 rows of two
// experts, n 1536, k 2048: 13 against 8); 64 rows an item where an expert has more than 16
// (64 rows: 41 against 37 with 16; 1024 rows: 47 and 46; with 32 rows an expert 69, where 16
// would read and convert every weight twice).
hipError_t launch_grouped_mm_few(const GroupedMm& g, int num_cus, hipStream_t s) {
  const bool swiglu = g.form == kMm4Swiglu, tall = g.rows > 16 * (int64_t)g.groups;
  const int oc = swiglu ? 16 : 32;
  const int64_t segments = g.rows / (tall ? 64 : 16) + std::min<int64_t>(g.groups, g.rows);
  const bool whole = segments * ((g.n_out + oc - 1) / oc) >= 4 * num_cus;
  const int wc = whole ? 4 * oc : oc;
  const int64_t items = segments * ((g.n_out + wc - 1) / wc);
  const unsigned blocks = (unsigned)std::min<int64_t>(items, 4 * num_cus);
  auto go = [&](auto kernel) {
    kernel<<<blocks, 256, 0, s>>>(g);
    return hipGetLastError();
  };
  return with_rows(g.dtype, [&](auto* t) {
    typedef std::remove_pointer_t<decltype(t)> T;
    if (g.form == kMm) {
      if constexpr (sizeof(T) == 2)
        return go(whole ? grouped_mm_few_kernel<T, false, false, 1, 1> : grouped_mm_few_kernel<T, false, false, 4, 1>);
      return hipErrorInvalidValue;
    }
    auto four_bit = [&](auto act) {
      constexpr bool S = decltype(act)::value;
      if (tall) return go(whole ? grouped_mm_few_kernel<T, true, S, 1, 4> : grouped_mm_few_kernel<T, true, S, 4, 4>);
      return go(whole ? grouped_mm_few_kernel<T, true, S, 1, 1> : grouped_mm_few_kernel<T, true, S, 4, 1>);
    };
    return swiglu ? four_bit(std::true_type{}) : four_bit(std::false_type{});
  });
}

}  // namespace moe
