// Activation checkpoints in 8 bits: pack, unpack, the SwiGLU that keeps its gate and up
// projections so, and the SwiGLU backward that reads them.
//
// A training step keeps the expert pre-activations g and u from the forward to the
// backward ([Review] section 4 trains the layer; which state a step keeps is not fixed
// by the pages). Rows are cut into blocks of 32 columns (the last one of a row may be
// shorter). With amax the largest magnitude in a block,
//   e = max(floor(log2 amax) - 6, -126),  q = clamp(rint(v 2^-e), -127, 127),
// the code q (int8) stands for q 2^e, and the block's scale byte is e + 127: float32
// exponent bits, so the scale and every product with it are exact and the codes do not
// depend on how they are computed. |v - q 2^e| <= 2^(e-1), or 2^e where |v| > 127.5 2^e
// is clamped; either is at most 2^-7 of the block's largest value (64 to 128 steps) while
// that is at least 2^-120. Below, where e stays -126, half a step is 2^-127: a block within
// 2^-127 becomes zeros.
// int8 steps are uniform, so a block's error goes by its largest value; an 8-bit float
// (4 significant bits) would be off by up to 2^-4 of that value itself. A block that
// holds a NaN or an infinity has scale byte 255 and codes 0 and stands for NaN.
//
// Every kernel moves C columns per lane and step, 8 or 16 (with_cols): a block is four or
// two adjacent lanes, whose maxima meet in quad permutations. All are bound by HBM.
#include <algorithm>
#include <type_traits>

#include "act8.hpp"
#include "common.hpp"
#include "kernels.hpp"
#include "rows.hpp"

namespace moe {

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ int64_t live_rows(const int32_t* n_rows, int64_t rows) {
  return n_rows ? min<int64_t>(max<int64_t>(n_rows[0], 0), rows) : rows;
}

// Scale bytes of a row (64 bits: cols may be any int32 multiple of 8, so cols + 31 is more
// than an int holds for the last of them).
__host__ __device__ __forceinline__ int64_t blocks_of(int cols) { return ((int64_t)cols + 31) / 32; }

// Largest of a value over the lanes of a block (two or four, inside a quad).
template <int C>
__device__ __forceinline__ uint32_t block_max(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true));  // lanes 1 0 3 2
  if (C == 8) v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true));  // lanes 2 3 0 1
  return v;
}

// The block's scale byte for C values per lane (lanes past the row hold zeros).
template <int C>
__device__ __forceinline__ uint32_t block_scale(const float* v) {
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < C; ++j) m = max(m, act8_magnitude(v[j]));
  return act8_scale(block_max<C>(m));
}

// C codes, stored and loaded at once.
template <int C>
using Codes = uint32_t __attribute__((ext_vector_type(C / 4)));

template <int C>
__device__ __forceinline__ void store_codes(uint8_t* p, const float* v, uint32_t scale) {
  Codes<C> q;
#pragma unroll
  for (int j = 0; j < C / 4; ++j) q[j] = act8_encode(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3], scale);
  *reinterpret_cast<Codes<C>*>(p) = q;
}

// C values q 2^e, exact (0 times the NaN block's infinite scale is NaN).
template <int C>
__device__ __forceinline__ void decode(Codes<C> c, uint32_t scale, float* v) {
  const float s = __uint_as_float(scale << 23);
#pragma unroll
  for (int j = 0; j < C; ++j) v[j] = (float)(int8_t)(c[j >> 2] >> (8 * (j & 3))) * s;
}

// C elements of a row, eight at a time.
template <int C, typename T>
__device__ __forceinline__ void load_cols(const T* p, float* v) {
#pragma unroll
  for (int j = 0; j < C; j += 8) load_row<8>(p + j, v + j);
}
template <int C, typename T>
__device__ __forceinline__ void store_cols(T* p, const float* v) {
#pragma unroll
  for (int j = 0; j < C; j += 8) store_row<8>(p + j, v + j);
}

// Where thread i of a launch works: rows of `padded` steps (whole blocks, so that a block's
// lanes stay together), the division by it as a multiplication (exact for i < 2^32).
struct RowMap {
  uint32_t padded;  // steps per row, rounded up to whole blocks
  uint32_t steps;   // steps per row
  uint64_t magic;   // floor(2^64 / padded) + 1
};
__device__ __forceinline__ void locate(const RowMap& m, uint32_t i, uint32_t& row, uint32_t& step) {
  const uint64_t lo = (uint64_t)i * (uint32_t)m.magic, hi = (uint64_t)i * (uint32_t)(m.magic >> 32);
  row = (uint32_t)((hi + (lo >> 32)) >> 32);
  step = i - row * m.padded;
}

// One step of C columns after another over the live rows, f(row, column, on); a lane off
// the row's end still takes part in its block. A workgroup takes kThreads consecutive
// steps at a time from a 64-bit base, so rows are counted from the base's row.
template <int C, typename F>
__device__ __forceinline__ void for_steps(const RowMap& m, int64_t rows, F&& f) {
  const int64_t total = rows * m.padded;
  for (int64_t base = (int64_t)blockIdx.x * kThreads; base < total; base += (int64_t)gridDim.x * kThreads) {
    const int64_t row0 = base / m.padded;
    uint32_t row, step;
    locate(m, (uint32_t)(base - row0 * m.padded) + threadIdx.x, row, step);
    if (row0 + row < rows) f(row0 + row, (int64_t)step * C, step < m.steps);
  }
}

// (16384 x 2048 bf16: 24 us, 102 MB at 4.2 TB/s with both ends of the kernel)
template <typename XT, int C>
__global__ void __launch_bounds__(kThreads)
act8_pack_kernel(const XT* __restrict__ x, int64_t ldx, const int32_t* __restrict__ n_rows, int64_t rows, int cols,
                 RowMap m, uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  const int64_t nb = blocks_of(cols);
  for_steps<C>(m, live_rows(n_rows, rows), [&](int64_t row, int64_t col, bool on) {
    float v[C] = {};
    if (on) load_cols<C>(x + row * ldx + col, v);
    const uint32_t s = block_scale<C>(v);
    if (on) store_codes<C>(codes + row * cols + col, v, s);
    if (on && (col & 31) == 0) scales[row * nb + col / 32] = (uint8_t)s;
  });
}

// (16384 x 2048 to bf16: 18 us, 102 MB at 5.8 TB/s, the codes partly still in the cache)
template <typename XT, int C>
__global__ void __launch_bounds__(kThreads)
act8_unpack_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                   const int32_t* __restrict__ n_rows, int64_t rows, int cols, RowMap m, XT* __restrict__ out,
                   int64_t ldo) {
  const int64_t nb = blocks_of(cols);
  for_steps<C>(m, live_rows(n_rows, rows), [&](int64_t row, int64_t col, bool on) {
    if (!on) return;
    float v[C];
    decode<C>(*reinterpret_cast<const Codes<C>*>(codes + row * cols + col), scales[row * nb + col / 32], v);
    store_cols<C>(out + row * ldo + col, v);
  });
}

// 1 / (1 + e^-z). FAST: the hardware's exponential and reciprocal, for 16-bit h, dg and du.
// The exponential's argument z log2 e is off by its own rounding, so the relative error
// grows with |z|: at most (1.5 |z| + 6) 2^-23, 2^-16 at z = -80 (half a step of bf16 is
// 2^-8, of half 2^-11). The backward's dw, a float32 sum, takes the sigmoid of the h it is
// summed from, so with 16-bit outputs its terms carry that error too.
template <bool FAST>
__device__ __forceinline__ float sigmoid(float z) {
  if constexpr (FAST) return __builtin_amdgcn_rcpf(1.0f + __expf(-z));
  return 1.0f / (1.0f + expf(-z));
}

// h and both checkpoints in one pass over g and u (32768 x 1536 bf16: 74 us, 406 MB at
// 5.5 TB/s, a copy's rate).
template <typename XT, int C>
__global__ void __launch_bounds__(kThreads)
swiglu_keep8_kernel(const XT* __restrict__ g, const XT* __restrict__ u, int64_t ld, const int32_t* __restrict__ n_rows,
                    int64_t rows, int F, RowMap m, XT* __restrict__ h, uint8_t* __restrict__ cg,
                    uint8_t* __restrict__ sg, uint8_t* __restrict__ cu, uint8_t* __restrict__ su) {
  const int64_t nb = blocks_of(F);
  for_steps<C>(m, live_rows(n_rows, rows), [&](int64_t row, int64_t col, bool on) {
    float z[C] = {}, v[C] = {};
    if (on) {
      load_cols<C>(g + row * ld + col, z);
      load_cols<C>(u + row * ld + col, v);
    }
    const uint32_t bz = block_scale<C>(z), bv = block_scale<C>(v);
    if (!on) return;
    store_codes<C>(cg + row * F + col, z, bz);
    store_codes<C>(cu + row * F + col, v, bv);
    if ((col & 31) == 0) {
      sg[row * nb + col / 32] = (uint8_t)bz;
      su[row * nb + col / 32] = (uint8_t)bv;
    }
    float o[C];
#pragma unroll
    for (int j = 0; j < C; ++j) o[j] = z[j] * sigmoid<sizeof(XT) == 2>(z[j]) * v[j];
    store_cols<C>(h + row * F + col, o);
  });
}

struct Bwd8 {
  const uint8_t *cg, *sg, *cu, *su;
  const int32_t* n_rows;
  const float* w_rows;
  const int32_t* row_slot;
  float* dw;
  int64_t n_slots, rows, ld;
  int F;
};

// C columns of the SwiGLU backward. Returns the sum of dh h over them.
template <int C, typename DT, typename OT>
__device__ __forceinline__ float swiglu_bwd8_step(const Bwd8& a, const DT* dh, OT* dg, OT* du, OT* h, int64_t nb,
                                                  int64_t row, int64_t col, float w) {
  float z[C], u[C], d[C], oh[C], dot = 0.0f;
  const int64_t at = row * a.F + col, b = row * nb + col / 32;
  const Codes<C> qz = *reinterpret_cast<const Codes<C>*>(a.cg + at), qu = *reinterpret_cast<const Codes<C>*>(a.cu + at);
  const uint32_t bz = a.sg[b], bu = a.su[b];
  load_cols<C>(dh + at, d);
  decode<C>(qz, bz, z);
  decode<C>(qu, bu, u);
#pragma unroll
  for (int j = 0; j < C; ++j) {
    const float s = sigmoid<sizeof(OT) == 2>(z[j]), act = z[j] * s, wd = w * d[j];
    oh[j] = act * u[j];
    dot = fmaf(d[j], oh[j], dot);
    z[j] = wd * u[j] * (s * (1.0f + z[j] * (1.0f - s)));  // dg
    u[j] = wd * act;                                      // du
  }
  store_cols<C>(dg + row * a.ld + col, z);
  store_cols<C>(du + row * a.ld + col, u);
  if (h) store_cols<C>(h + at, oh);
  return dot;
}

// Rows without weight gradients: steps of 8 columns, any row to any lane (16384 x 1536,
// float32 dh, bf16 out: 56 us, 303 MB at 5.4 TB/s).
template <typename DT, typename OT, int C>
__global__ void __launch_bounds__(kThreads)
swiglu_bwd8_kernel(Bwd8 a, RowMap m, const DT* __restrict__ dh, OT* __restrict__ dg, OT* __restrict__ du,
                   OT* __restrict__ h) {
  const int64_t nb = blocks_of(a.F);
  for_steps<C>(m, live_rows(a.n_rows, a.rows), [&](int64_t row, int64_t col, bool on) {
    if (on) swiglu_bwd8_step<C>(a, dh, dg, du, h, nb, row, col, a.w_rows ? a.w_rows[row] : 1.0f);
  });
}

// Rows with weight gradients dw = <dh, h>, TPR threads per row whose sums are added in a
// fixed order. A wavefront (64) for most; four of them (256) for few long rows, which
// leave most of the chip's wavefronts free (bf16, us with one against four: 1 x 1536 5.4
// and 3.4, 1024 x 1536 7.6 and 6.3, 64 x 14336 35 and 11; but 4096 x 1536 14.2 and 15.3,
// 32768 x 1536 96 and 106); for rows shorter than a wavefront's 512 columns (TPR 0) tpr
// lanes, the least power of two from 8 on that covers the row's steps (65536 x 64 51 and
// 12 us, 65536 x 256 63 and 38). rows is the tensors' capacity, the only count the host
// has: few live rows of a large capacity keep one wavefront each.
constexpr int64_t kFewRows = 2048;
template <typename DT, typename OT, int TPR, int C>
__global__ void __launch_bounds__(kThreads)
swiglu_bwd8_row_kernel(Bwd8 a, int tpr, const DT* __restrict__ dh, OT* __restrict__ dg, OT* __restrict__ du,
                       OT* __restrict__ h) {
  constexpr int kWaves = kThreads / kWave;
  __shared__ float part[kWaves];
  const int group = TPR ? TPR : tpr;  // threads per row, a power of two
  const int rpw = kThreads / group;   // rows per workgroup
  const int sub = threadIdx.x & (group - 1);
  const int64_t n = live_rows(a.n_rows, a.rows), nb = blocks_of(a.F);
  for (int64_t row0 = (int64_t)blockIdx.x * rpw; row0 < n; row0 += (int64_t)gridDim.x * rpw) {
    const int64_t row = row0 + threadIdx.x / group;
    float dot = 0.0f;
    if (row < n) {
      const float w = a.w_rows ? a.w_rows[row] : 1.0f;
      for (int64_t col = sub * C; col < a.F; col += group * C)
        dot += swiglu_bwd8_step<C>(a, dh, dg, du, h, nb, row, col, w);
    }
    for (int o = min(group, kWave) / 2; o > 0; o >>= 1) dot += __shfl_xor(dot, o, kWave);
    if (TPR > kWave) {
      if (threadIdx.x % kWave == 0) part[threadIdx.x / kWave] = dot;
      __syncthreads();
      if (sub == 0)
        for (int i = 1; i < kWaves; ++i) dot += part[i];
      __syncthreads();
    }
    if (row < n && sub == 0) {
      const int64_t to = a.row_slot ? a.row_slot[row] : row;
      if (to >= 0 && to < a.n_slots) a.dw[to] = dot;
    }
  }
}

RowMap row_map(int cols, int C) {
  RowMap m;
  m.steps = (uint32_t)(cols / C);
  m.padded = (m.steps + 32 / C - 1) / (32 / C) * (32 / C);
  m.magic = ~uint64_t(0) / m.padded + 1;
  return m;
}
// Workgroups over the steps of all rows (the live rows are only known on the device).
unsigned grid_of(int64_t rows, const RowMap& m) {
  return (unsigned)std::max<int64_t>(1, std::min<int64_t>((rows * m.padded + kThreads - 1) / kThreads, 1 << 20));
}
// Calls f with the step width of an encoding kernel: 16 columns for 16-bit tensors whose
// rows of codes start at multiples of 16, if they are many: a lane then stores 16 bytes of
// codes at once (bf16, us with 8 and 16: pack 32768 x 1536 32.6 and 28.9, 4096 x 768 3.7 and 3.3, but
// 256 x 1536 2.5 and 2.7, with half the wavefronts; keep8 77 and 74, 7.5 and 7.2, 3.0 and
// 3.4). Float32 gains nothing (24.6 and 24.5; keep8 65 and 70), and the decoding kernels,
// whose stores are wide anyway, lose (unpack 30.3 and 32.3, SwiGLU backward 91 and 98).
// rows is the capacity here too: few live rows of a large one take 16 columns, at the small
// sizes' loss above.
template <typename XT, typename F>
hipError_t with_cols(int64_t rows, int cols, F&& f) {
  if constexpr (sizeof(XT) == 2)
    if (cols % 16 == 0 && rows * cols >= (1 << 20)) return f(std::integral_constant<int, 16>{});
  return f(std::integral_constant<int, 8>{});
}

}  // namespace

hipError_t launch_act8_pack(int dtype, const void* x, int64_t ldx, const int32_t* n_rows, int64_t rows, int cols,
                            void* codes, void* scales, hipStream_t s) {
  return with_rows(dtype, [&](auto* t) {
    typedef std::remove_pointer_t<decltype(t)> XT;
    return with_cols<XT>(rows, cols, [&](auto c) {
      constexpr int C = decltype(c)::value;
      const RowMap m = row_map(cols, C);
      act8_pack_kernel<XT, C><<<grid_of(rows, m), kThreads, 0, s>>>(static_cast<const XT*>(x), ldx, n_rows, rows, cols,
                                                                    m, static_cast<uint8_t*>(codes),
                                                                    static_cast<uint8_t*>(scales));
      return hipGetLastError();
    });
  });
}

hipError_t launch_act8_unpack(int dtype, const void* codes, const void* scales, const int32_t* n_rows, int64_t rows,
                              int cols, void* out, int64_t ldo, hipStream_t s) {
  return with_rows(dtype, [&](auto* t) {
    typedef std::remove_pointer_t<decltype(t)> XT;
    constexpr int C = 8;
    const RowMap m = row_map(cols, C);
    act8_unpack_kernel<XT, C><<<grid_of(rows, m), kThreads, 0, s>>>(
        static_cast<const uint8_t*>(codes), static_cast<const uint8_t*>(scales), n_rows, rows, cols, m,
        static_cast<XT*>(out), ldo);
    return hipGetLastError();
  });
}

hipError_t launch_swiglu_keep8(const SwigluKeep8Args& a, hipStream_t s) {
  return with_rows(a.dtype, [&](auto* t) {
    typedef std::remove_pointer_t<decltype(t)> XT;
    return with_cols<XT>(a.rows, a.F, [&](auto c) {
      constexpr int C = decltype(c)::value;
      const RowMap m = row_map(a.F, C);
      swiglu_keep8_kernel<XT, C><<<grid_of(a.rows, m), kThreads, 0, s>>>(
          static_cast<const XT*>(a.g), static_cast<const XT*>(a.u), a.ld, a.n_rows, a.rows, a.F, m,
          static_cast<XT*>(a.h), static_cast<uint8_t*>(a.codes_g), static_cast<uint8_t*>(a.scales_g),
          static_cast<uint8_t*>(a.codes_u), static_cast<uint8_t*>(a.scales_u));
      return hipGetLastError();
    });
  });
}

hipError_t launch_swiglu_bwd8(const SwigluBwd8Args& a, hipStream_t s) {
  const Bwd8 b{static_cast<const uint8_t*>(a.codes_g), static_cast<const uint8_t*>(a.scales_g),
               static_cast<const uint8_t*>(a.codes_u), static_cast<const uint8_t*>(a.scales_u),
               a.n_rows, a.w_rows, a.row_slot, a.dw, a.n_slots, a.rows, a.ld, a.F};
  return with_rows(a.dh_dtype, [&](auto* t) {
    return with_rows(a.out_dtype, [&](auto* o) {
      typedef std::remove_pointer_t<decltype(t)> DT;
      typedef std::remove_pointer_t<decltype(o)> OT;
      const DT* dh = static_cast<const DT*>(a.dh);
      OT *dg = static_cast<OT*>(a.dg), *du = static_cast<OT*>(a.du), *h = static_cast<OT*>(a.h);
      constexpr int C = 8;
      if (a.dw) {
        int tpr = 8;
        while (tpr < kWave && tpr * C < a.F) tpr *= 2;
        if (a.F > kWave * C && a.rows <= kFewRows) tpr = kThreads;
        const int rpw = kThreads / tpr;
        const unsigned blocks = (unsigned)std::min<int64_t>((a.rows + rpw - 1) / rpw, 1 << 20);
        auto go = [&](auto kernel) { kernel<<<blocks, kThreads, 0, s>>>(b, tpr, dh, dg, du, h); };
        if (tpr == kThreads) go(swiglu_bwd8_row_kernel<DT, OT, kThreads, C>);
        else if (tpr == kWave) go(swiglu_bwd8_row_kernel<DT, OT, kWave, C>);
        else go(swiglu_bwd8_row_kernel<DT, OT, 0, C>);
      } else {
        const RowMap m = row_map(a.F, C);
        swiglu_bwd8_kernel<DT, OT, C><<<grid_of(a.rows, m), kThreads, 0, s>>>(b, m, dh, dg, du, h);
      }
      return hipGetLastError();
    });
  });
}

}  // namespace moe
