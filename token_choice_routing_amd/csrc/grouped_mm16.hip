// Grouped products of 16-bit rows and weights on the matrix cores (forms as in
// grouped_mm.hip): tiles of BM x BN outputs, the reduction 32 at a time.
#include <algorithm>

#include "grouped_mm.hpp"
#include "rows.hpp"

namespace moe {

namespace {

constexpr int kBK = 32, kStages = 4;
constexpr uint32_t kPast = 0xfffffff0u;     // byte offset past every resource: reads zero, touches nothing
constexpr uint32_t kRecords = 0xffffff00u;  // (lanes that read anything are bounded by their own tests)

typedef short s16x4_t __attribute__((ext_vector_type(4)));

template <typename T>
__device__ __forceinline__ f32x16_t mfma16(bf16x8_t j, bf16x8_t i, f32x16_t c) {
  if constexpr (std::is_same<T, bf16_t>::value)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(j, i, c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_t, j), __builtin_bit_cast(f16x8_t, i), c, 0,
                                                  0, 0);
}

// v_permlane32_swap_b32: lane half 0 gets (a, a of the lane 32 on), half 1 (b of the lane 32
// back, b).
__device__ __forceinline__ u32x2_t swap_lane_halves(uint32_t a, uint32_t b) {
#if defined(__HIP_DEVICE_COMPILE__)
  const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
  return u32x2_t{r[0], r[1]};
#else
  return u32x2_t{a, b};
#endif
}

// A 4-element column of a K-major stage by the transposing LDS read: within each 16-lane
// block lane i receives element i % 4 of the 4-element pieces that lanes 4 j + i / 4 (j =
// 0..3) address.
__device__ __forceinline__ s16x4_t read_tr(const char* __restrict__ p) {
#if defined(__HIP_DEVICE_COMPILE__)
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4_t*)p);
#else
  (void)p;
  return s16x4_t{};
#endif
}

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

template <typename T, int FORM, int BM, int BN, int WM, int WN>
__global__ void __launch_bounds__(64 * WM * WN) __attribute__((amdgpu_waves_per_eu(2, 2)))
grouped_mm16_kernel(GroupedMm g) {
  constexpr int NW = WM * WN, FM = BM / WM / 32, FN = BN / WN / 32;
  constexpr bool KI = FORM == kMmWgrad, KJ = FORM != kMm;  // K-major operands (the reduction runs over their rows)
  constexpr int PI = BM / 16 / NW, PJ = BN / 16 / NW;      // 1 KB pieces of a stage that a wavefront loads
  constexpr int PL = PI + PJ;
  constexpr int STAGE = (BM + BN) * kBK * 2;               // bytes
  __shared__ Segments sg;
  extern __shared__ __attribute__((aligned(16))) char smem[];  // [kStages][I region, J region]
  const int I = KI ? g.n_out : 0, J = FORM == kMm ? g.n_out : g.k_dim;
  const int nt = (J + BN - 1) / BN;
  const int total = build_segments(sg, g.offsets, g.groups, g.rows, BM, nt, I);
  const int lane = threadIdx.x & (kWave - 1), wave = uniform(threadIdx.x / kWave);
  const int wm = wave / WN, wn = wave % WN;  // (the wavefronts of a SIMD have different rows)
  const int half = lane >> 5, l32 = lane & 31;

  // Tiles (expert, column tile, row tile), an eighth of the list for each XCD.
  const int xcd = blockIdx.x & 7, slot = blockIdx.x >> 3, per = gridDim.x >> 3;
  const int first = (int)((int64_t)xcd * total / 8), count = (int)((int64_t)(xcd + 1) * total / 8) - first;

  struct Item {
    int e, start, i0, iv, j0, jv, klen;  // valid rows and columns of the tile; length of the reduction
  };
  auto locate = [&](int it) {
    Item w;
    const int t = first + it;
    w.e = uniform(segment_of(sg, g.groups, t));
    const int local = t - uniform(sg.prefix[w.e]);
    const int len = uniform(sg.len[w.e]);
    w.start = uniform(sg.start[w.e]);
    const int extent = KI ? I : len;
    const int mt = (extent + BM - 1) / BM;
    w.j0 = local / mt * BN;
    w.i0 = local % mt * BM;
    w.iv = min(BM, extent - w.i0);
    w.jv = min(BN, J - w.j0);
    w.klen = KI ? len : FORM == kMmDgrad ? g.n_out : g.k_dim;
    return w;
  };

  // This lane's share of a piece. Row-major: 16 rows of 32, the lane's 16-byte chunk lc of
  // row lane / 4 (chunks XOR-ed with (row / 4) % 4 against bank conflicts). K-major: 512 / B
  // K rows of B columns, 64-byte groups XOR-ed with the K row.
  const int lc = (lane & 3) ^ (lane >> 4);
  auto krow = [&](int piece, int B) { return piece * (512 / B) + lane / (B / 8); };
  auto kcol = [&](int kr, int B) {
    const int p = lane % (B / 8);
    return ((p & 3) | (((p >> 2) ^ (kr & 3)) << 2)) * 8;
  };

  // ---- the stream of K tiles, kStages ahead of the products, item after item
  const T* isrc = nullptr;
  const T* jsrc = nullptr;
  uint32_t ioff[PI], joff[PJ];
  int lit = slot, lkt = 0, lnk = 0, lklen = 0, lstart = 0;
  int64_t istep = 0, jstep = 0;
  const uint32_t lda2 = (uint32_t)g.lda * 2;
  auto open_item = [&]() {
    // the next item with anything to reduce over
    lkt = 0;
    lnk = 0;
    lklen = 0;
    while (lit < count) {
      const Item w = locate(lit);
      lit += per;
      if (w.klen == 0) continue;
      lklen = w.klen;
      lnk = (w.klen + kBK - 1) / kBK;
      lstart = w.start;
      const int64_t ild = FORM == kMm ? g.lda : g.ldy;
      const T* ibase = static_cast<const T*>(FORM == kMm ? g.a : g.dy);
      const bool gather = FORM == kMm && g.a_rows;
      if (!gather) ibase += (int64_t)(w.start + (KI ? 0 : w.i0)) * ild + (KI ? w.i0 : 0);
      isrc = uniform_ptr(ibase);
      istep = KI ? kBK * ild : kBK;
#pragma unroll
      for (int p = 0; p < PI; ++p) {
        if constexpr (KI) {
          const int kr = krow(wave + NW * p, BM), c = kcol(kr, BM);
          ioff[p] = c < w.iv ? (uint32_t)(kr * ild + c) * 2u : kPast;
        } else {
          const int r = 16 * (wave + NW * p) + (lane >> 2);
          int64_t row = r;
          if (gather) row = min<int64_t>(max<int64_t>(g.a_rows[w.start + w.i0 + min(r, w.iv - 1)], 0), g.a_nrows - 1);
          ioff[p] = r < w.iv ? (uint32_t)(row * ild + lc * 8) * 2u : kPast;
        }
      }
      const T* jbase;
      if (FORM == kMmWgrad) jbase = static_cast<const T*>(g.a) + (g.a_rows ? 0 : (int64_t)w.start * g.lda) + w.j0;
      else if (FORM == kMmDgrad) jbase = static_cast<const T*>(g.w) + (int64_t)w.e * g.n_out * g.k_dim + w.j0;
      else jbase = static_cast<const T*>(g.w) + ((int64_t)w.e * g.n_out + w.j0) * g.k_dim;
      jsrc = uniform_ptr(jbase);
      const int64_t jld = FORM == kMmWgrad ? g.lda : g.k_dim;
      jstep = KJ ? (FORM == kMmWgrad && g.a_rows ? 0 : kBK * jld) : kBK;
#pragma unroll
      for (int p = 0; p < PJ; ++p) {
        if constexpr (KJ) {
          const int kr = krow(wave + NW * p, BN), c = kcol(kr, BN);
          const bool rowless = FORM == kMmWgrad && g.a_rows;  // the row is added at each tile
          joff[p] = c < w.jv ? (uint32_t)((rowless ? 0 : kr * jld) + c) * 2u : kPast;
        } else {
          const int r = 16 * (wave + NW * p) + (lane >> 2);
          joff[p] = r < w.jv ? (uint32_t)(r * jld + lc * 8) * 2u : kPast;
        }
      }
      return;
    }
  };
  auto issue = [&](int st) {
    if (lkt == lnk) open_item();
    char* stage = smem + st * STAGE;
    const auto ri = buffer_rsrc(isrc, kRecords), rj = buffer_rsrc(jsrc, kRecords);
    const int k0 = lkt * kBK;
    const bool whole = k0 + kBK <= lklen;
#pragma unroll
    for (int p = 0; p < PI; ++p) {
      const int piece = wave + NW * p;
      const int k = k0 + (KI ? krow(piece, BM) : lc * 8);
      buffer_load_lds16(ri, whole || k < lklen ? ioff[p] : kPast, reinterpret_cast<bf16_t*>(stage + piece * 1024));
    }
#pragma unroll
    for (int p = 0; p < PJ; ++p) {
      const int piece = wave + NW * p;
      const int k = k0 + (KJ ? krow(piece, BN) : lc * 8);
      uint32_t off = joff[p];
      if (FORM == kMmWgrad && g.a_rows && lnk) {
        const int64_t row = g.a_rows[lstart + min(k, lklen - 1)];
        off += (uint32_t)min<int64_t>(max<int64_t>(row, 0), g.a_nrows - 1) * lda2;
        if (joff[p] == kPast) off = kPast;
      }
      buffer_load_lds16(rj, whole || k < lklen ? off : kPast,
                        reinterpret_cast<bf16_t*>(stage + BM * kBK * 2 + piece * 1024));
    }
    isrc = uniform_ptr(isrc + istep);
    jsrc = uniform_ptr(jsrc + jstep);
    if (lkt < lnk) ++lkt;
  };

  // ---- fragments: per 16-wide K step FN J blocks and FM I blocks of 32
  uint32_t iaddr[KI ? FM : 2], jaddr[KJ ? FN : 2];
  {
    const int s16 = lane & 15;
    const int kl = 8 * half + (s16 >> 2), nl = 16 * ((lane >> 4) & 1) + 4 * (s16 & 3);
    if constexpr (KI) {
#pragma unroll
      for (int b = 0; b < FM; ++b) iaddr[b] = (uint32_t)(kl * BM + (((wm * FM + b) ^ (kl & 3)) * 32) + nl) * 2;
    } else {
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
        iaddr[ks] = (uint32_t)((wm * FM * 32 + l32) * kBK + (((2 * ks + half) ^ ((l32 >> 2) & 3)) << 3)) * 2;
    }
    if constexpr (KJ) {
#pragma unroll
      for (int b = 0; b < FN; ++b)
        jaddr[b] = (uint32_t)(BM * kBK + kl * BN + (((wn * FN + b) ^ (kl & 3)) * 32) + nl) * 2;
    } else {
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
        jaddr[ks] = (uint32_t)(BM * kBK + (wn * FN * 32 + l32) * kBK + (((2 * ks + half) ^ ((l32 >> 2) & 3)) << 3)) * 2;
    }
  }
  struct Frags {
    bf16x8_t j[FN], i[FM];
  };
  auto column = [&](const char* p, int ks, int B) {
    const s16x4_t lo = read_tr(p + ks * 16 * B * 2), hi = read_tr(p + (ks * 16 + 4) * B * 2);
    return __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  };
  auto read = [&](int st, int ks, Frags& f) {
    const char* stage = smem + st * STAGE;
#pragma unroll
    for (int b = 0; b < FN; ++b) {
      if constexpr (KJ) f.j[b] = column(stage + jaddr[b], ks, BN);
      else f.j[b] = *reinterpret_cast<const bf16x8_t*>(stage + jaddr[ks] + b * 32 * kBK * 2);
    }
#pragma unroll
    for (int b = 0; b < FM; ++b) {
      if constexpr (KI) f.i[b] = column(stage + iaddr[b], ks, BM);
      else f.i[b] = *reinterpret_cast<const bf16x8_t*>(stage + iaddr[ks] + b * 32 * kBK * 2);
    }
  };

  if (slot >= count) return;
#pragma unroll
  for (int s = 0; s < kStages; ++s) issue(s);
  wait_vmcnt<(kStages - 1) * PL>();
  stage_barrier();
  int st = 0;
  for (int it = slot; it < count; it += per) {
    const Item w = locate(it);
    const bool on = wm * FM * 32 < w.iv && wn * FN * 32 < w.jv;
    f32x16_t acc[FN][FM];
#pragma unroll
    for (int f = 0; f < FN; ++f)
#pragma unroll
      for (int b = 0; b < FM; ++b) acc[f][b] = f32x16_t{};
    auto multiply = [&](const Frags& f) {
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int b = 0; b < FM; ++b) acc[j][b] = mfma16<T>(f.j[j], f.i[b], acc[j][b]);
    };
    const int nk = (w.klen + kBK - 1) / kBK;
    Frags f0, f1;
    if (on && nk) read(st, 0, f0);
    for (int kt = 0; kt < nk; ++kt) {
      const int next = (st + 1) & (kStages - 1);
      if (on) {
        read(st, 1, f1);
        multiply(f0);
      }
      // the next tile of the stream has landed, and every wavefront is done with this one
      wait_vmcnt<(kStages - 2) * PL>();
      stage_barrier();
      issue(st);
      if (on) {
        if (kt + 1 < nk) read(next, 0, f0);
        multiply(f1);
      }
      st = next;
    }
    if (!on) continue;
#pragma unroll
    for (int b = 0; b < FM; ++b) {
      const int r = wm * FM * 32 + b * 32 + l32;
      if (r >= w.iv) continue;
      const int64_t row = KI ? ((int64_t)w.e * g.n_out + w.i0 + r) * g.k_dim : (int64_t)(w.start + w.i0 + r) * g.ldo;
#pragma unroll
      for (int f = 0; f < FN; ++f) {
        const int c0 = w.j0 + wn * FN * 32 + f * 32;
        f32x16_t v = acc[f][b];
        if (KI && g.add) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int col = c0 + 8 * q + 4 * half;
            if (col >= J) continue;
            const f32x4_t a = *reinterpret_cast<const f32x4_t*>(g.add + row + col);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[4 * q + j] += a[j];
          }
        }
        if (g.out_dtype == MOE_F32) {
          float* out = static_cast<float*>(g.out) + row;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int col = c0 + 8 * q + 4 * half;
            if (col < J) *reinterpret_cast<f32x4_t*>(out + col) = f32x4_t{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
          }
          continue;
        }
        uint32_t p[8];
        if (g.out_dtype == MOE_BF16) {
#pragma unroll
          for (int q = 0; q < 8; ++q) p[q] = cvt_bf16x2(v[2 * q], v[2 * q + 1]);
        } else {
#pragma unroll
          for (int q = 0; q < 8; ++q) p[q] = pack_f16x2(v[2 * q], v[2 * q + 1]);
        }
        // lane halves exchanged: 16 neighbouring columns a lane
        uint16_t* out = static_cast<uint16_t*>(g.out) + row;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const u32x2_t x = swap_lane_halves(p[2 * q], p[2 * q + 4]), y = swap_lane_halves(p[2 * q + 1], p[2 * q + 5]);
          const int col = c0 + 16 * half + 8 * q;
          if (col < J) *reinterpret_cast<u32x4_t*>(out + col) = u32x4_t{x[0], y[0], x[1], y[1]};
        }
      }
    }
  }
  wait_vmcnt<0>();  // the stream's last loads land before the workgroup's LDS is given away
}

template <typename T, int BM, int BN, int WM, int WN>
hipError_t launch_tiles(const GroupedMm& g, int num_cus, hipStream_t s) {
  constexpr size_t lds = (size_t)kStages * (BM + BN) * kBK * 2;
  const int J = g.form == kMm ? g.n_out : g.k_dim;
  const int64_t nt = (J + BN - 1) / BN;
  const int64_t mt = g.form == kMmWgrad ? (int64_t)g.groups * ((g.n_out + BM - 1) / BM) : g.rows / BM + g.groups;
  const int64_t slots = (int64_t)num_cus * std::max<int>(1, (int)((160 * 1024) / (lds + sizeof(Segments))));
  const unsigned blocks = (unsigned)(std::min<int64_t>(slots, mt * nt + 7) / 8 * 8);
  auto go = [&](auto kernel) {
    (void)hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize,
                              (int)lds);
    kernel<<<blocks, 64 * WM * WN, lds, s>>>(g);
    return hipGetLastError();
  };
  switch (g.form) {
    case kMm: return go(grouped_mm16_kernel<T, kMm, BM, BN, WM, WN>);
    case kMmDgrad: return go(grouped_mm16_kernel<T, kMmDgrad, BM, BN, WM, WN>);
    case kMmWgrad: return go(grouped_mm16_kernel<T, kMmWgrad, BM, BN, WM, WN>);
  }
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_grouped_mm16(const GroupedMm& g, int num_cus, hipStream_t s) {
  return g.dtype == MOE_BF16 ? launch_tiles<bf16_t, 256, 256, 2, 4>(g, num_cus, s)
                             : launch_tiles<half_t, 256, 256, 2, 4>(g, num_cus, s);
}

}  // namespace moe
