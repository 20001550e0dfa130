// Products of rows in expert order with their expert's weights, over segments of any
// length (the grouped GEMM of the paper review "Improving MoE Compute Efficiency by
// Composing Weight and Data Sparsity", section 3 "implementation", as plain products with
// gradients, for experts of one's own):
//   product          out[p] = W[e] a[src(p)]           reduces over k_dim
//   data gradient    da[p] = W[e]^T dy[p]              reduces over n_out
//   weight gradient  dW[e] = add[e] + sum_p dy[p] a[src(p)]^T   reduces over the rows of e
// Each is C[i][j] = sum_k A[i][k] B[j][k] on the matrix cores, in tiles of BM x BN outputs and
// 64 bytes of a row (32 16-bit elements or 16 float32 ones) of the reduction at a time.
//
// 256 x 256 on eight wavefronts of 128 x 64: the largest whose sums and two sets of fragments
// fit the registers of two wavefronts a SIMD (208 of 256), and four stages the LDS (128 KB). A
// wavefront reads half a stage's fragments while it multiplies the other half, with one barrier
// a stage; the loads run four stages ahead and on into the next tiles. 8192^3 bf16: 860-920 us
// (1.20-1.28 PF; the library's product of this layout 670-711, of row-major B 790-875). 32889 rows of 64 experts, 22 to 2794 each, 1536 x
// 2048: product 256 us, 262 of gathered rows; data gradient 236; weight gradient (float32) 303, 324
// of gathered rows, 577 added to an earlier one (460 to 558 rows each: 250 and 257, 236, 296 and
// 308, 521). What bounds them there: the matrix pipe is busy 40-44% of the time; weights that come
// from memory once (product 229 us with equal experts of 512 rows, 201 with one expert), partly
// filled row tiles and the last round of tiles; in the weight gradient the 805 MB of stores (182
// us without them), and with an addend a load, a wait and a store for every 16 bytes of a lane.
#include <algorithm>

#include "grouped_mm.hpp"
#include "rows.hpp"

namespace moe {

namespace {

constexpr uint32_t kPast = 0xfffffff0u;     // byte offset past every resource: reads zero, touches nothing
constexpr uint32_t kRecords = 0xffffff00u;  // (lanes that read anything are bounded by their own tests)

constexpr int kBand = 8;  // row tiles that share a column panel in turn (8192^3: 1265 us without, 917 so)

typedef short s16x4_t __attribute__((ext_vector_type(4)));

// One step of a 32 x 32 block: 16 bytes of a J row and an I row a lane, lane half h holding the
// step's elements of its half. 16-bit: one product 16 deep. float32: four, 2 deep, element s of
// both halves in product s.
template <typename T>
__device__ __forceinline__ f32x16_t multiply_block(u32x4_t j, u32x4_t i, f32x16_t c) {
  if constexpr (std::is_same<T, float>::value) {
    const f32x4_t x = __builtin_bit_cast(f32x4_t, j), y = __builtin_bit_cast(f32x4_t, i);
#pragma unroll
    for (int s = 0; s < 4; ++s) c = __builtin_amdgcn_mfma_f32_32x32x2f32(x[s], y[s], c, 0, 0, 0);
    return c;
  } else if constexpr (std::is_same<T, bf16_t>::value) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, j), __builtin_bit_cast(bf16x8_t, i), c,
                                                   0, 0, 0);
  } else {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_t, j), __builtin_bit_cast(f16x8_t, i), c, 0,
                                                  0, 0);
  }
}

// A 4-element column of a K-major stage by the transposing LDS read: within each 16-lane
// block lane i receives element i % 4 of the 4-element pieces that lanes 4 j + i / 4 (j =
// 0..3) address. Without the __restrict__ the compiler cannot tell the read from the loads into
// LDS that are in flight and waits for all of them first; with it the read's own waits alone are
// left (the kernel waits for a stage's loads itself, before the barrier that opens the stage).
__device__ __forceinline__ s16x4_t read_tr(const char* __restrict__ p) {
#if defined(__HIP_DEVICE_COMPILE__)
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4_t*)p);
#else
  (void)p;
  return s16x4_t{};
#endif
}

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// Calls f with n as a constant (0 <= n <= N, the same in every lane).
template <int N, typename F>
__device__ __forceinline__ void deal(int n, F&& f) {
  if constexpr (N == 0) f(std::integral_constant<int, 0>{});
  else if (n >= N) f(std::integral_constant<int, N>{});
  else deal<N - 1>(n, f);
}

// ROWS: a weight gradient whose a is read through a_rows (then rows > 0).
template <typename T, int FORM, bool ROWS, int BM, int BN, int WM, int WN, int S>
__global__ void __launch_bounds__(64 * WM * WN) __attribute__((amdgpu_waves_per_eu(2, 2)))
grouped_mm_tiles_kernel(GroupedMm g) {
  constexpr int ES = sizeof(T), EC = 16 / ES, kBK = 64 / ES;  // bytes an element; elements of 16 bytes, of a stage's row
  constexpr int NW = WM * WN, FM = BM / WM / 32, FN = BN / WN / 32;
  constexpr bool KI = FORM == kMmWgrad, KJ = FORM != kMm;  // K-major operands (the reduction runs over their rows)
  constexpr int PI = BM / 16 / NW, PJ = BN / 16 / NW;      // 1 KB pieces of a stage that a wavefront loads
  constexpr int PL = PI + PJ;
  constexpr int STAGE = (BM + BN) * 64;                    // bytes
  __shared__ Segments sg;
  extern __shared__ __attribute__((aligned(16))) char smem[];  // [S][I region, J region]
  const int I = KI ? g.n_out : 0, J = FORM == kMm ? g.n_out : g.k_dim;
  const int nt = (J + BN - 1) / BN;
  const int total = build_segments(sg, g.offsets, g.groups, g.rows, BM, nt, I);
  const int lane = threadIdx.x & (kWave - 1), wave = uniform(threadIdx.x / kWave);
  const int wm = wave / WN, wn = wave % WN;  // (the wavefronts of a SIMD have different rows)
  const int half = lane >> 5, l32 = lane & 31;

  // Tiles (expert, band of row tiles, column tile, row tile), an eighth of the list (of a weight
  // gradient's: of the work) for each XCD: the tiles it runs at once share weight panels and row panels in its L2.
  const int xcd = blockIdx.x & 7, slot = blockIdx.x >> 3, per = gridDim.x >> 3;
  const int first = uniform(KI ? work_share(sg, g.groups, total, xcd) : (int)((int64_t)xcd * total / 8));
  const int count = uniform(KI ? work_share(sg, g.groups, total, xcd + 1) : (int)((int64_t)(xcd + 1) * total / 8)) - first;

  // (one tile a workgroup needs no order: it costs 1 us)
  const bool ordered = KI && count > per;
  if (ordered) largest_first(sg, g.groups, first, first + count);

  struct Item {
    int e, start, i0, iv, j0, jv, klen;  // valid rows and columns of the tile; length of the reduction
  };
  auto locate = [&](int it) __attribute__((always_inline)) {
    Item w;
    const int t = ordered ? it : first + it;
    const int at = uniform(segment_of(sg, g.groups, t));
    w.e = ordered ? uniform(sg.order[at]) : at;
    const int local = t - uniform(sg.prefix[at]) + (ordered ? uniform(sg.skip[at]) : 0);
    const int len = uniform(sg.len[w.e]);
    w.start = uniform(sg.start[w.e]);
    const int extent = KI ? I : len;
    const int mt = (extent + BM - 1) / BM;
    const int band = local / (kBand * nt), in = local - band * kBand * nt;
    const int high = min(kBand, mt - band * kBand);
    w.j0 = in / high * BN;
    const int tile = band * kBand + in % high, blocks = (extent + 31) / 32;
    w.i0 = (int)((int64_t)tile * blocks / mt) * 32;
    w.iv = min((int)((int64_t)(tile + 1) * blocks / mt) * 32, extent) - w.i0;
    w.jv = min(BN, J - w.j0);
    w.klen = KI ? len : FORM == kMmDgrad ? g.n_out : g.k_dim;
    return w;
  };

  // This lane's share of a piece. Row-major: 16 rows of 64 bytes, the lane's 16-byte chunk lc of
  // row lane / 4 (chunks XOR-ed with (row / 4) % 4 against bank conflicts). K-major: K rows of B
  // columns, 32-column groups XOR-ed with the K row (16-bit, whose reads take four K rows at
  // once) or its half of the stage (float32, whose reads take one of each half).
  const int lc = (lane & 3) ^ (lane >> 4);
  auto krow = [&](int piece, int B) { return piece * (1024 / (B * ES)) + lane / (B * ES / 16); };
  auto kswap = [&](int kr) { return ES == 2 ? kr & 3 : (kr >> 3) & 1; };
  auto kcol = [&](int kr, int B) {
    constexpr int GC = 32 / EC;  // chunks of a 32-column group
    const int p = lane % (B * ES / 16);
    return (p % GC + ((p / GC) ^ kswap(kr)) * GC) * EC;
  };

  // ---- the stream of K tiles, S ahead of the products, item after item
  const T* isrc = nullptr;
  const T* jsrc = nullptr;
  uint32_t ioff[PI], joff[PJ];
  int lit = slot, lkt = 0, lnk = 0, lklen = 0, lstart = 0;
  int64_t istep = 0, jstep = 0;
  const uint32_t lda_bytes = (uint32_t)g.lda * ES;
  // Gathered rows of the reduction: the rows that the wavefront's pieces of
  // the next K tile hold (the same in every lane, read as scalars a tile ahead: vector loads
  // return in order, so one would wait for every tile in flight).
  constexpr int KPP = KJ ? 1024 / (BN * ES) : 1;
  int32_t idx[PJ][KPP];
  const int last_row = (int)g.a_nrows - 1;  // ((a_nrows + 1) rows fit in 32 bits)
  typedef const __attribute__((address_space(4))) int32_t* scalar_rows;
  const scalar_rows a_rows = (scalar_rows)(uintptr_t)g.a_rows;
  auto fetch_rows = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int p = 0; p < PJ; ++p)
#pragma unroll
      for (int q = 0; q < KPP; ++q) {
        const int k = min(lkt * kBK + (wave + NW * p) * KPP + q, max(lklen - 1, 0));
        idx[p][q] = a_rows[(uint32_t)uniform(lstart + k)];
      }
  };
  // Rows of the next item's I pieces in a gathered product, read an item ahead.
  const bool gather = FORM == kMm && g.a_rows;
  int32_t nrow[PI];
  auto fetch_next = [&]() __attribute__((always_inline)) {
    if (!gather || lit >= count) return;
    const Item w = locate(lit);
#pragma unroll
    for (int p = 0; p < PI; ++p)
      nrow[p] = g.a_rows[w.start + w.i0 + min(16 * (wave + NW * p) + (lane >> 2), w.iv - 1)];
  };
  fetch_next();
  auto open_item = [&]() __attribute__((always_inline)) {
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
      if (!gather) ibase += (int64_t)(w.start + (KI ? 0 : w.i0)) * ild + (KI ? w.i0 : 0);
      isrc = uniform_ptr(ibase);
      istep = KI ? kBK * ild : kBK;
#pragma unroll
      for (int p = 0; p < PI; ++p) {
        if constexpr (KI) {
          const int kr = krow(wave + NW * p, BM), c = kcol(kr, BM);
          ioff[p] = c < w.iv ? (uint32_t)(kr * ild + c) * ES : kPast;
        } else {
          const int r = 16 * (wave + NW * p) + (lane >> 2);
          int64_t row = r;
          if (gather) row = min<int64_t>(max<int64_t>(nrow[p], 0), g.a_nrows - 1);
          ioff[p] = r < w.iv ? (uint32_t)(row * ild + lc * EC) * ES : kPast;
        }
      }
      const T* jbase;
      if (FORM == kMmWgrad) jbase = static_cast<const T*>(g.a) + (ROWS ? 0 : (int64_t)w.start * g.lda) + w.j0;
      else if (FORM == kMmDgrad) jbase = static_cast<const T*>(g.w) + (int64_t)w.e * g.n_out * g.k_dim + w.j0;
      else jbase = static_cast<const T*>(g.w) + ((int64_t)w.e * g.n_out + w.j0) * g.k_dim;
      jsrc = uniform_ptr(jbase);
      const int64_t jld = FORM == kMmWgrad ? g.lda : g.k_dim;
      jstep = KJ ? (ROWS ? 0 : kBK * jld) : kBK;
#pragma unroll
      for (int p = 0; p < PJ; ++p) {
        if constexpr (KJ) {
          const int kr = krow(wave + NW * p, BN), c = kcol(kr, BN);
          // (of gathered rows: the row is added at each tile)
          joff[p] = c < w.jv ? (uint32_t)((ROWS ? 0 : kr * jld) + c) * ES : kPast;
        } else {
          const int r = 16 * (wave + NW * p) + (lane >> 2);
          joff[p] = r < w.jv ? (uint32_t)(r * jld + lc * EC) * ES : kPast;
        }
      }
      if constexpr (ROWS) fetch_rows();
      fetch_next();
      return;
    }
  };
  auto issue = [&](int st) __attribute__((always_inline)) {
    if (lkt == lnk) open_item();
    char* stage = smem + st * STAGE;
    const auto ri = buffer_rsrc(isrc, kRecords), rj = buffer_rsrc(jsrc, kRecords);
    const int k0 = lkt * kBK;
    const bool whole = k0 + kBK <= lklen;
#pragma unroll
    for (int p = 0; p < PI; ++p) {
      const int piece = wave + NW * p;
      const int k = k0 + (KI ? krow(piece, BM) : lc * EC);
      buffer_load_lds16(ri, whole || k < lklen ? ioff[p] : kPast, reinterpret_cast<bf16_t*>(stage + piece * 1024));
    }
#pragma unroll
    for (int p = 0; p < PJ; ++p) {
      const int piece = wave + NW * p;
      const int k = k0 + (KJ ? krow(piece, BN) : lc * EC);
      uint32_t off = joff[p];
      if constexpr (ROWS) {
        // (of four the compiler would otherwise make an array in scratch memory, indexed by lane: a
        // load and a wait for every tile in flight)
        int row = idx[p][0];
#pragma unroll
        for (int q = 1; q < KPP; ++q)
          row = lane / (BN * ES / 16) >= q ? (KPP > 2 ? opaque_v(idx[p][q]) : idx[p][q]) : row;
        off = off == kPast ? kPast : off + (uint32_t)min(max(row, 0), last_row) * lda_bytes;
      }
      buffer_load_lds16(rj, whole || k < lklen ? off : kPast,
                        reinterpret_cast<bf16_t*>(stage + BM * 64 + piece * 1024));
    }
    isrc = uniform_ptr(isrc + istep);
    jsrc = uniform_ptr(jsrc + jstep);
    if (lkt < lnk) ++lkt;
  };
  // Before each issue(), and as early as the loop has it: the scalar loads of gathered rows. The
  // fragments read before are waited for first: scalar loads return in no order, so an LDS wait
  // behind them would be one for everything.
  auto before_issue = [&]() __attribute__((always_inline)) {
    if constexpr (ROWS) {
      __builtin_amdgcn_s_waitcnt((63 & 15) | ((63 >> 4) << 14) | (7 << 4));  // lgkmcnt(0)
      fetch_rows();  // (past an item's end: some row of it; the next item's are read when it is opened)
    }
  };

  // ---- fragments: per half of a stage's K FN J blocks and FM I blocks of 32, 16 bytes a lane.
  // Row-major: chunk 2 ks + h (16-bit) or ks + 2 h (float32) of the lane's row for half h of the
  // lanes. K-major, 16-bit: two transposing reads; float32: an element of each of four K rows.
  auto chunk_of = [&](int ks) { return ES == 2 ? 2 * ks + half : ks + 2 * half; };
  uint32_t iaddr[KI ? FM : 2], jaddr[KJ ? FN : 2];
  {
    const int s16 = lane & 15;
    const int kl = 8 * half + (ES == 2 ? s16 >> 2 : 0), nl = ES == 2 ? 16 * ((lane >> 4) & 1) + 4 * (s16 & 3) : l32;
    if constexpr (KI) {
#pragma unroll
      for (int b = 0; b < FM; ++b) iaddr[b] = (uint32_t)(kl * BM + ((b * WM + wm) ^ kswap(kl)) * 32 + nl) * ES;
    } else {
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
        iaddr[ks] = (uint32_t)((wm * 32 + l32) * 64 + ((chunk_of(ks) ^ ((l32 >> 2) & 3)) << 4));
    }
    if constexpr (KJ) {
#pragma unroll
      for (int b = 0; b < FN; ++b)
        jaddr[b] = (uint32_t)(BM * 64 + (kl * BN + ((wn * FN + b) ^ kswap(kl)) * 32 + nl) * ES);
    } else {
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
        jaddr[ks] = (uint32_t)(BM * 64 + (wn * FN * 32 + l32) * 64 + ((chunk_of(ks) ^ ((l32 >> 2) & 3)) << 4));
    }
  }
  struct Frags {
    u32x4_t j[FN], i[FM];
  };
  auto column = [&](const char* p, int ks, int B) __attribute__((always_inline)) {
    if constexpr (ES == 2) {
      const s16x4_t lo = read_tr(p + ks * 16 * B * 2), hi = read_tr(p + (ks * 16 + 4) * B * 2);
      return __builtin_bit_cast(u32x4_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
      u32x4_t v;
#pragma unroll
      for (int s = 0; s < 4; ++s) v[s] = *reinterpret_cast<const uint32_t*>(p + (4 * ks + s) * B * 4);
      return v;
    }
  };
  auto read = [&](auto blocks, int st, int ks, Frags& f) __attribute__((always_inline)) {
    constexpr int NB = decltype(blocks)::value;
    const char* stage = smem + st * STAGE;
#pragma unroll
    for (int b = 0; b < FN; ++b) {
      if constexpr (KJ) f.j[b] = column(stage + jaddr[b], ks, BN);
      else f.j[b] = *reinterpret_cast<const u32x4_t*>(stage + jaddr[ks] + b * 32 * 64);
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      if constexpr (KI) f.i[b] = column(stage + iaddr[b], ks, BM);
      else f.i[b] = *reinterpret_cast<const u32x4_t*>(stage + iaddr[ks] + b * WM * 32 * 64);
    }
  };

  // ---- outputs. In the products' layout a lane holds 16 columns of one row; a store of 16
  // bytes a lane would touch 32 rows, and a CU then writes 37 GB/s. Turned round in LDS (8 rows
  // of 128 bytes a 1 KB piece, 16-byte chunks XOR-ed with the row), eight lanes store 128
  // bytes of a row: 115 GB/s. Rows and columns past the tile's get an offset past the resource.
  auto out_at = [&](const Item& w) __attribute__((always_inline)) {  // the tile's first element
    return KI ? ((int64_t)w.e * g.n_out + w.i0) * g.k_dim + w.j0 : (int64_t)(w.start + w.i0) * g.ldo + w.j0;
  };
  auto piece_at = [&](char* stage, int i) __attribute__((always_inline)) {
    if (PL < 4) return smem + S * STAGE + (4 * wave + i) * 1024;  // (too few pieces: LDS of its own)
    return stage + (i < PI ? wave + NW * i : BM / 16 + wave + NW * (i - PI)) * 1024;
  };
  // type: the output's. float32 goes 32 columns at a time; 16-bit types 64, but 32 with ADD, whose
  // addends are float32, and where the wavefront has no more.
  auto store = [&](auto type, auto added, auto stream, const Item& w, const f32x16_t (&acc)[FN][FM],
                   char* stage) __attribute__((always_inline)) {
    typedef decltype(type) OT;
    constexpr bool ADD = decltype(added)::value, WIDE = std::is_same<OT, float>::value || ADD;
    constexpr int C = WIDE || FN == 1 ? 1 : 2;  // 32-column blocks at a time
    constexpr int CL = WIDE ? 4 : 8;            // columns a lane reads back
    constexpr int kPolicy = decltype(stream)::value ? 2 : 0;  // nt: not kept in the caches
    const int lane = opaque_v((int)threadIdx.x) & (kWave - 1), half = lane >> 5, l32 = lane & 31;
    const int r8 = lane >> 3, c8 = lane & 7;
    char* const mine[4] = {piece_at(stage, 0), piece_at(stage, 1), piece_at(stage, 2), piece_at(stage, 3)};
    // this lane's row of a 32-row block, and the piece rows it reads back
    char* const put = (l32 < 8 ? mine[0] : l32 < 16 ? mine[1] : l32 < 24 ? mine[2] : mine[3]) + (l32 & 7) * 128;
    const int get = r8 * 128 + ((c8 ^ r8) << 4);
    const int64_t at = out_at(w);
    const auto ro = buffer_rsrc(uniform_ptr(static_cast<const OT*>(g.out) + at), kRecords);
    const auto ra = buffer_rsrc(uniform_ptr(g.add + (ADD ? at : 0)), kRecords);
    const uint32_t ld = (uint32_t)(KI ? g.k_dim : g.ldo);
    auto pack = [](float x, float y) {
      return std::is_same<OT, half_t>::value ? pack_f16x2(x, y) : cvt_bf16x2(x, y);
    };
#pragma unroll
    for (int b = 0; b < FM; ++b) {
#pragma unroll
      for (int f = 0; f < FN; f += C) {
#pragma unroll
        for (int h = 0; h < C; ++h)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const f32x16_t& v = acc[f + h][b];
            const f32x4_t x = {v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
            if constexpr (WIDE)
              *reinterpret_cast<f32x4_t*>(put + (((2 * q + half) ^ (l32 & 7)) << 4)) = x;
            else
              *reinterpret_cast<u32x2_t*>(put + (((4 * h + q) ^ (l32 & 7)) << 4) + 8 * half) =
                  u32x2_t{pack(x[0], x[1]), pack(x[2], x[3])};
          }
        const int c = wn * FN * 32 + f * 32 + CL * c8;
        const bool cols = CL * c8 < 32 * C;  // (half a line of 16-bit outputs where FN is 1)
        u32x4_t x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const u32x4_t*>(mine[i] + get);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = (b * WM + wm) * 32 + 8 * i + r8;
          const bool in = cols && r < w.iv && c < w.jv;
          const uint32_t el = (uint32_t)r * ld + (uint32_t)c;
          if constexpr (ADD) {
            const f32x4_t y =
                __builtin_bit_cast(f32x4_t, __builtin_amdgcn_raw_buffer_load_b128(ra, in ? el * 4u : kPast, 0, 0));
            const f32x4_t z = __builtin_bit_cast(f32x4_t, x[i]) + y;
            if constexpr (std::is_same<OT, float>::value)
              x[i] = __builtin_bit_cast(u32x4_t, z);
            else
              x[i] = u32x4_t{pack(z[0], z[1]), pack(z[2], z[3]), 0, 0};
          }
          const uint32_t off = in ? el * (uint32_t)sizeof(OT) : kPast;
          if constexpr (ADD && sizeof(OT) == 2)
            __builtin_amdgcn_raw_buffer_store_b64(u32x2_t{x[i][0], x[i][1]}, ro, off, 0, kPolicy);
          else
            __builtin_amdgcn_raw_buffer_store_b128(x[i], ro, off, 0, kPolicy);
        }
      }
    }
  };
  auto store_as = [&](const Item& w, const f32x16_t (&acc)[FN][FM], char* stage) __attribute__((always_inline)) {
    // A weight gradient is larger than the caches and written once: its lines are not kept, if
    // they are whole ones (64 x 1536 x 2048 float32: 305 -> 280 us; with rows of 3104 bytes
    // kept ones take 50 us and others 99).
    auto typed = [&](auto type) __attribute__((always_inline)) {
      if constexpr (KI) {
        const bool whole = (g.k_dim * sizeof(type)) % 128 == 0 && reinterpret_cast<uintptr_t>(g.out) % 128 == 0;
        if (g.add) store(type, std::true_type{}, std::false_type{}, w, acc, stage);
        else if (sizeof(type) == 4 && whole) store(type, std::false_type{}, std::true_type{}, w, acc, stage);
        else store(type, std::false_type{}, std::false_type{}, w, acc, stage);
      } else {
        store(type, std::false_type{}, std::false_type{}, w, acc, stage);
      }
    };
    if (g.out_dtype == MOE_F32) typed(float{});
    else if (g.out_dtype == MOE_BF16) typed(bf16_t{});
    else typed(half_t{});
  };
  // The output of an expert without rows: what is added, or zeros.
  auto store_zero = [&](const Item& w) {
    for (int i = lane; i < FM * 32 * FN * 4; i += kWave) {
      const int r = (i / (FN * 4 * 32) * WM + wm) * 32 + i / (FN * 4) % 32, col = w.j0 + wn * FN * 32 + i % (FN * 4) * 8;
      if (r >= w.iv || col >= J) continue;
      const int64_t at = ((int64_t)w.e * g.n_out + w.i0 + r) * g.k_dim + col;
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = 0.0f;
      if (KI && g.add) load_row<8>(g.add + at, v);
      if (g.out_dtype == MOE_F32) store_row<8>(static_cast<float*>(g.out) + at, v);
      else if (g.out_dtype == MOE_BF16) store_row<8>(static_cast<bf16_t*>(g.out) + at, v);
      else store_row<8>(static_cast<half_t*>(g.out) + at, v);
    }
  };

  if (slot >= count) return;
#pragma unroll 1  // (opening an item is long code, which should stay in the instruction cache)
  for (int s = 0; s < S; ++s) {
    before_issue();
    issue(s);
  }
  wait_vmcnt<(S - 1) * PL>();
  stage_barrier();
  int st = 0;
  for (int it = slot; it < count; it += per) {
    const Item w = locate(it);
    // 32-row blocks of the tile, dealt out to the WM wavefronts of a column: a short tile
    // leaves every SIMD the same share
    const int mine = wn * FN * 32 < w.jv ? max(0, ((w.iv + 31) / 32 - wm + WM - 1) / WM) : 0;
    f32x16_t acc[FN][FM];
#pragma unroll
    for (int f = 0; f < FN; ++f)
#pragma unroll
      for (int b = 0; b < FM; ++b) acc[f][b] = f32x16_t{};
    const int nk = (w.klen + kBK - 1) / kBK;
    auto reduce = [&](auto blocks) __attribute__((always_inline)) {
      constexpr int NB = decltype(blocks)::value;
      auto multiply = [&](const Frags& f) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int b = 0; b < NB; ++b) acc[j][b] = multiply_block<T>(f.j[j], f.i[b], acc[j][b]);
      };
      Frags f0, f1;
      if (NB && nk) read(blocks, st, 0, f0);
      for (int kt = 0; kt < nk; ++kt) {
        const int next = st + 1 == S ? 0 : st + 1;
        before_issue();
        if (NB) {
          read(blocks, st, 1, f1);
          multiply(f0);
        }
        // the next tile of the stream has landed, and every wavefront is done with this one
        wait_vmcnt<(S - 2) * PL>();
        stage_barrier();
        if (kt + 1 < nk) {
          issue(st);
          if (NB) read(blocks, next, 0, f0);
        }
        if (NB) multiply(f1);
        if (kt + 1 < nk) st = next;
      }
    };
    deal<FM>(mine, reduce);
    // The stage of the last tile is free: each wavefront turns its outputs round in the pieces
    // of it that it loads itself, then loads them.
    if (mine && nk) store_as(w, acc, smem + st * STAGE);
    if (mine && !nk) store_zero(w);  // (only a weight gradient has such items)
    if (nk) {
      issue(st);
      st = st + 1 == S ? 0 : st + 1;
    }
  }
  wait_vmcnt<0>();  // the stream's last loads land before the workgroup's LDS is given away
}

template <typename T, int BM, int BN, int WM, int WN, int S>
hipError_t launch_tiles(const GroupedMm& g, int num_cus, hipStream_t s) {
  constexpr size_t lds = (size_t)S * (BM + BN) * 64 + ((BM + BN) / 16 / (WM * WN) < 4 ? WM * WN * 4096 : 0);
  const int J = g.form == kMm ? g.n_out : g.k_dim;
  const int64_t nt = (J + BN - 1) / BN;
  const int64_t mt = g.form == kMmWgrad ? (int64_t)g.groups * ((g.n_out + BM - 1) / BM) : g.rows / BM + g.groups;
  const int64_t slots = (int64_t)num_cus * std::max<int>(1, (int)((160 * 1024) / (lds + sizeof(Segments))));
  const unsigned blocks = (unsigned)(std::min<int64_t>(slots, mt * nt + 7) / 8 * 8);
  auto go = [&](auto kernel) {
    if (lds > 64 * 1024)
      (void)hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize,
                                (int)lds);
    kernel<<<blocks, 64 * WM * WN, lds, s>>>(g);
    return hipGetLastError();
  };
  switch (g.form) {
    case kMm: return go(grouped_mm_tiles_kernel<T, kMm, false, BM, BN, WM, WN, S>);
    case kMmDgrad: return go(grouped_mm_tiles_kernel<T, kMmDgrad, false, BM, BN, WM, WN, S>);
    case kMmWgrad:
      return g.a_rows && g.rows ? go(grouped_mm_tiles_kernel<T, kMmWgrad, true, BM, BN, WM, WN, S>)
                                : go(grouped_mm_tiles_kernel<T, kMmWgrad, false, BM, BN, WM, WN, S>);
  }
  return hipErrorInvalidValue;
}

// Tiles of 128 x 128 (two workgroups a CU) where 256 x 256 would leave CUs idle, and for a
// product of so few rows that it reads its weights once whatever the tile. us with 256 and 128:
//   product 1024 rows of 8 experts, 1536 x 2048: 34 and 25; 1024 of 64: 105 and 88, 9600 of 64:
//   126 and 137, 32768 of 8, 1024 x 1024: 72 and 98
//   data gradient 1024 of 8: 29 and 21, 9600 of 64: 97 and 141 (and 73 and 78 at 1024 of 64)
//   weight gradient 32768 of 8, 1024 x 1024 (128 tiles of 256 x 256): 100 and 80; 16384 of 1, 1536 x
//   2048: 346 and 177; 16372 of 64, 768 x 1024 (768 tiles): 60 and 103
// float32: 64 x 64 where 128 x 128 would. us with 128 and 64: 896 rows of 16 experts, 520 x 264: 16
// and 11, data gradient 27 and 17; 8192 of 8, 768 x 1024: 130 and 128, data gradient 105 and 132;
// weight gradient 4096 of 1, 1024 x 1024 (64 tiles): 285 and 103; 32970 of 64, 768 x 1024: 420 and 577
template <typename T>
hipError_t launch_for(const GroupedMm& g, int num_cus, hipStream_t s) {
  const int J = g.form == kMm ? g.n_out : g.k_dim;
  auto tiles = [&](int b) {
    return (g.form == kMmWgrad ? (int64_t)g.groups * ((g.n_out + b - 1) / b) : g.rows / b + g.groups) * ((J + b - 1) / b);
  };
  if constexpr (std::is_same<T, float>::value) {
    const bool small = tiles(128) < num_cus;
    return small ? launch_tiles<T, 64, 64, 2, 2, 4>(g, num_cus, s) : launch_tiles<T, 128, 128, 2, 2, 4>(g, num_cus, s);
  } else {
    const bool small = g.form == kMmWgrad
                           ? tiles(256) < 2 * num_cus
                           : tiles(256) < num_cus || (g.form == kMm && g.rows <= 64 * (int64_t)g.groups);
    return small ? launch_tiles<T, 128, 128, 2, 2, 4>(g, num_cus, s) : launch_tiles<T, 256, 256, 2, 4, 4>(g, num_cus, s);
  }
}

}  // namespace

hipError_t launch_grouped_mm(const GroupedMm& g, int num_cus, hipStream_t s) {
  // Few rows. us there and in the tiles, 2048 x 1536, bf16:
  //   2 rows of 8 experts 8 and 16, 12 of each of 8: 14 and 17 (768 x 1024, 16 of each of 16: 11 and 14)
  //   64 experts, 1, 4, 8 or 16 rows each: 75 and 80, 76 and 82, 79 and 85, 85 and 87
  //   as many rows by Zipf's law: 39 and 42, 71 and 79, 99 and 89, 118 and 105; all of one expert: 22
  //   and 19, 23 and 21, 39 and 21, 70 and 24 (128 experts, 16 on average: 133 and 28)
  // The weights of an expert are read again for every 16 of its rows there, and only the device
  // knows which expert has how many. So: up to 4 rows an expert on average, which keeps what even
  // rows gain and bounds what one large expert costs, or up to 256 rows of 16 on average.
  const bool few = g.form == kMm && g.dtype != MOE_F32 && g.rows <= 16 * (int64_t)g.groups &&
                   g.rows <= std::max<int64_t>(4 * (int64_t)g.groups, 256);
  if (few || g.form == kMm4 || g.form == kMm4Swiglu) return launch_grouped_mm_few(g, num_cus, s);
  return with_rows(g.dtype, [&](auto* t) { return launch_for<std::remove_pointer_t<decltype(t)>>(g, num_cus, s); });
}

}  // namespace moe
