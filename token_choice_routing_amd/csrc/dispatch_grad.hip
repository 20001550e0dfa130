// Token rows to and from expert order for experts outside the layer call: the
// weighted way back for rows of any storage type, its gradient, and the gradient of
// the way there.
//
// Paper review "Improving MoE Compute Efficiency by Composing Weight and Data
// Sparsity", section 3, core formula y_t = E_shared(x_t) + sum_k g_k E_{i_k}(x_t) and
// the "implementation" paragraph (slots sorted by expert, null slots cut off). With
// r_tk the row a slot contributes (an expert row of a real slot, the null source of a
// copy or constant null slot, nothing otherwise):
//   combine            y_t = ys_t + sum_k w_tk r_tk
//   its gradient       dr_p = w_tk dy_t (p the slot's position), dw_tk = <dy_t, r_tk>,
//                      null source: sum over null slots of w_tk dy_t
//   gather's gradient  dx_t = add_t + sum over real slots of dx_p
// Every sum runs in float32 in slot order and is rounded once. All of them only move
// rows: they are bound by HBM, at a few operations per element.
#include <algorithm>
#include <type_traits>

#include "common.hpp"
#include "kernels.hpp"
#include "rows.hpp"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kCols = 8;   // columns per lane
constexpr int kSpan = kWave * kCols;  // columns per wavefront
// Slots whose rows are loaded before the first is used. Eight take the registers of
// half the wavefronts (combine at 16384 x 2048, 8 slots a quarter real: 62 us against 53).
constexpr int kGroup = 4;

// Position of a slot: a row of y_perm, or what stands in for one.
constexpr int kNullSlot = -1, kNoSlot = -2;

// y[t] = shared[t] + sum over slots of w r, in slot order (fmaf, one rounding). One
// wavefront per token and span of kSpan columns: the token's positions and weights are
// read once by lanes 0..K-1 and broadcast, and every row's load is in flight before the
// first is added. A wavefront with two or four spans of a token reads the positions less
// often but holds fewer loads in flight over the chip (16384 x 2048, 8 slots a quarter
// real, bf16: 50.7 us at 5.3 TB/s with one span, 52.8 with two, 73 with four).
// WEIGHTED false: every weight is 1.
template <typename RT, typename AT, typename ET, bool WEIGHTED>
__global__ void __launch_bounds__(kThreads)
slot_sum_kernel(const RT* __restrict__ rows, const int32_t* __restrict__ slot_pos,
                const float* __restrict__ topk_w, const AT* shared, const ET* __restrict__ null_src,
                int64_t null_stride, ET* y, int64_t T, int K, int d, int64_t max_rows, int spans) {
  const int lane = threadIdx.x & (kWave - 1);
  const int64_t wave = (int64_t)blockIdx.x * (kThreads / kWave) + threadIdx.x / kWave;
  const int64_t nwaves = (int64_t)gridDim.x * (kThreads / kWave);
  const int64_t units = T * spans;
  for (int64_t unit = wave; unit < units; unit += nwaves) {
    const int64_t t = unit / spans;
    const int c = (int)(unit - t * spans) * kSpan + lane * kCols;
    const bool on = c < d;
    int my_p = kNoSlot;
    float my_w = 1.0f;
    if (lane < K) {
      my_p = slot_pos[t * K + lane];
      if (WEIGHTED) my_w = topk_w[t * K + lane];
      if (my_p == kNullSlot ? !null_src : (my_p < 0 || my_p >= max_rows)) my_p = kNoSlot;
    }
    float acc[kCols], nul[kCols];
#pragma unroll
    for (int j = 0; j < kCols; ++j) acc[j] = nul[j] = 0.0f;
    if (on) {
      if (shared) load_row<kCols>(shared + t * d + c, acc);
      if (null_src) load_row<kCols>(null_src + t * null_stride + c, nul);
    }
    uint64_t todo = ballot(my_p != kNoSlot);
    while (todo) {
      int p[kGroup];
      float w[kGroup];
      RawRow<RT, kCols> r[kGroup];
#pragma unroll
      for (int g = 0; g < kGroup; ++g) {
        p[g] = kNoSlot;
        if (todo) {
          const int k = __builtin_ctzll(todo);
          todo &= todo - 1;
          p[g] = __builtin_amdgcn_readlane(my_p, k);
          w[g] = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(my_w), k));
          if (p[g] >= 0 && on) r[g].load(rows + (int64_t)p[g] * d + c);
        }
      }
#pragma unroll
      for (int g = 0; g < kGroup; ++g) {
        if (p[g] >= 0) {
#pragma unroll
          for (int j = 0; j < kCols; ++j)
            acc[j] = WEIGHTED ? fmaf(w[g], r[g][j], acc[j]) : acc[j] + r[g][j];
        } else if (p[g] == kNullSlot) {
#pragma unroll
          for (int j = 0; j < kCols; ++j) acc[j] = fmaf(w[g], nul[j], acc[j]);
        }
      }
    }
    if (on) store_row<kCols>(y + t * d + c, acc);
  }
}

// Sum over the wavefront, the same in every lane: rows of 16 lanes by permutations
// inside them, then the rows' sums passed up (lane 63 holds the total).
template <int CTRL, int ROWS>
__device__ __forceinline__ float add_dpp(float v) {
  return v + __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), CTRL, ROWS, 0xF, false));
}
__device__ __forceinline__ float wave_sum(float v) {
  v = add_dpp<0xB1, 0xF>(v);   // lanes 1 0 3 2
  v = add_dpp<0x4E, 0xF>(v);   // lanes 2 3 0 1
  v = add_dpp<0x141, 0xF>(v);  // mirrored in halves of a row
  v = add_dpp<0x140, 0xF>(v);  // mirrored in a row
  v = add_dpp<0x142, 0xA>(v);  // lane 15 of rows 0, 2 into rows 1, 3
  v = add_dpp<0x143, 0xC>(v);  // lane 31 into rows 2, 3
  return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), 63));
}

// Gradient of the constant null expert's vector, sum over tokens of (sum of the null
// slots' weights) dy_t: float32 sums over chunks of tokens, one wavefront per chunk and
// 256 columns, then a float64 sum of the chunks in a fixed order. Chunks of 16 tokens (the
// whole gradient in us, 8 slots a quarter real, with 8, 16 and 64: 200 x 1024 6.2, 6.5 and 10.7;
// 2047 x 1024 10.3, 10.8 and 16.2; 16384 x 2048 91, 84 and 85: shorter ones write more
// partial sums, longer ones leave few wavefronts with long chains).
constexpr int kNullCols = 4;
constexpr int kNullChunk = 16;
// The units (chunk, columns) of wavefront `wave` of nwaves.
template <typename ET>
__device__ __forceinline__ void null_vector_partial(const ET* __restrict__ dy, const int32_t* __restrict__ slot_pos,
                                                    const float* __restrict__ topk_w, int64_t T, int K, int d,
                                                    int64_t wave, int64_t nwaves, float* __restrict__ part) {
  const int lane = threadIdx.x & (kWave - 1);
  const int spans = (d + kWave * kNullCols - 1) / (kWave * kNullCols);
  const int64_t chunks = (T + kNullChunk - 1) / kNullChunk;
  for (int64_t unit = wave; unit < chunks * spans; unit += nwaves) {
    const int64_t at = unit / spans, t0 = at * kNullChunk;
    const int n = (int)min<int64_t>(kNullChunk, T - t0);
    const int c = (int)(unit - at * spans) * kWave * kNullCols + lane * kNullCols;
    float my_w = 0.0f;  // lane i: token t0 + i
    bool any = false;
    if (lane < n)
      for (int k = 0; k < K; ++k)
        if (slot_pos[(t0 + lane) * K + k] == kNullSlot) {
          my_w += topk_w[(t0 + lane) * K + k];
          any = true;
        }
    float acc[kNullCols] = {0.0f, 0.0f, 0.0f, 0.0f};
    constexpr int kAhead = 8;
    for (uint64_t todo = ballot(any); todo;) {
      RawRow<ET, kNullCols> g[kAhead];
      float w[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        w[i] = 0.0f;
        g[i].zero();
        if (todo) {
          const int k = __builtin_ctzll(todo);
          todo &= todo - 1;
          w[i] = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(my_w), k));
          if (c < d) g[i].load(dy + (t0 + k) * d + c);
        }
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
#pragma unroll
        for (int j = 0; j < kNullCols; ++j) acc[j] = fmaf(w[i], g[i][j], acc[j]);
    }
    if (c < d) store_row<kNullCols>(part + at * d + c, acc);
  }
}

// The combine's gradient: WPT wavefronts per token, each with every WPT-th span of
// kSpan columns, whose parts of the slots' products meet in LDS. One wavefront per token
// holds the whole row's loads in registers and so fewer of them over the chip (16384 x
// 2048, 8 slots a quarter real, bf16: 106 us, 80 us with two slots at a time, 67 us so).
// The constant null vector's sums over token chunks run in workgroups of the same launch.
template <typename RT, typename ET, int WPT>
__global__ void __launch_bounds__(kThreads)
combine_bwd_kernel(const ET* __restrict__ dy, const RT* __restrict__ y_perm, const int32_t* __restrict__ slot_pos,
                   const float* __restrict__ topk_w, const ET* __restrict__ null_src, int64_t null_stride,
                   RT* __restrict__ dy_perm, float* __restrict__ w_perm, int32_t* __restrict__ row_slot,
                   float* __restrict__ dtopk_w, float* __restrict__ dnull, int64_t T, int K, int d,
                   int64_t max_rows, unsigned blocks, float* __restrict__ null_part) {
  constexpr int kTokens = kThreads / kWave / WPT;  // tokens per workgroup
  if (blockIdx.x >= blocks) {  // the workgroups behind those of the tokens
    constexpr int kWaves = kThreads / kWave;
    null_vector_partial(dy, slot_pos, topk_w, T, K, d, (int64_t)(blockIdx.x - blocks) * kWaves + threadIdx.x / kWave,
                        (int64_t)(gridDim.x - blocks) * kWaves, null_part);
    return;
  }
  __shared__ float part[kThreads / kWave][MOE_MAX_TOPK];
  // (the wavefront's number through readfirstlane: its token and span are then uniform
  // values to the compiler, 69.6 -> 67.3 us)
  const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int sub = wave % WPT;
  const bool dots = y_perm && dtopk_w;
  for (int64_t t0 = (int64_t)blockIdx.x * kTokens; t0 < T; t0 += (int64_t)blocks * kTokens) {
    const int64_t t = t0 + wave / WPT;
    int my_p = kNoSlot;
    float my_w = 0.0f, my_dot = 0.0f;  // lane k: slot k
    if (t < T && lane < K) {
      my_p = slot_pos[t * K + lane];
      my_w = topk_w[t * K + lane];
      if (my_p != kNullSlot && (my_p < 0 || my_p >= max_rows)) my_p = kNoSlot;
      if (my_p >= 0 && sub == 0) {
        if (w_perm) w_perm[my_p] = my_w;
        if (row_slot) row_slot[my_p] = (int32_t)(t * K + lane);
      }
    }
    const uint64_t reals = ballot(my_p >= 0), nulls = ballot(my_p == kNullSlot);
    float wn = 0.0f;  // sum of the null slots' weights
    if (dnull)
      for (uint64_t m = nulls; m; m &= m - 1)
        wn += __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(my_w), __builtin_ctzll(m)));
    for (int c0 = sub * kSpan; t < T && c0 < d; c0 += WPT * kSpan) {
      const int c = c0 + lane * kCols;
      const bool on = c < d;
      RawRow<ET, kCols> g, nul;
      g.zero();
      nul.zero();
      if (on) g.load(dy + t * d + c);
      const bool null_dot = null_src && dtopk_w && nulls;
      if (null_dot && on) nul.load(null_src + t * null_stride + c);
      // the expert rows, kGroup slots at a time
      for (uint64_t todo = dy_perm || dots ? reals : 0; todo;) {
        int p[kGroup], k[kGroup];
        float w[kGroup];
        RawRow<RT, kCols> r[kGroup];
#pragma unroll
        for (int i = 0; i < kGroup; ++i) {
          p[i] = kNoSlot;
          r[i].zero();
          if (todo) {
            k[i] = __builtin_ctzll(todo);
            todo &= todo - 1;
            p[i] = __builtin_amdgcn_readlane(my_p, k[i]);
            w[i] = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(my_w), k[i]));
            if (dots && on) r[i].load(y_perm + (int64_t)p[i] * d + c);
          }
        }
        if (dy_perm && on) {
#pragma unroll
          for (int i = 0; i < kGroup; ++i) {
            if (p[i] < 0) continue;
            float o[kCols];
#pragma unroll
            for (int j = 0; j < kCols; ++j) o[j] = w[i] * g[j];
            store_row<kCols>(dy_perm + (int64_t)p[i] * d + c, o);
          }
        }
        if (dots) {
#pragma unroll
          for (int i = 0; i < kGroup; ++i) {
            if (p[i] < 0) continue;
            float dot = 0.0f;
#pragma unroll
            for (int j = 0; j < kCols; ++j) dot = fmaf(g[j], r[i][j], dot);
            dot = wave_sum(dot);
            if (lane == k[i]) my_dot += dot;
          }
        }
      }
      // the null slots share one product; the copied token gets their weights' sum times dy
      if (null_dot) {
        float dot = 0.0f;
#pragma unroll
        for (int j = 0; j < kCols; ++j) dot = fmaf(g[j], nul[j], dot);
        dot = wave_sum(dot);
        if (my_p == kNullSlot) my_dot += dot;
      }
      if (dnull && on) {
        float o[kCols];
#pragma unroll
        for (int j = 0; j < kCols; ++j) o[j] = nulls ? wn * g[j] : 0.0f;
        store_row<kCols>(dnull + t * d + c, o);
      }
    }
    if (!dtopk_w) continue;
    if (WPT > 1) {
      if (lane < MOE_MAX_TOPK) part[wave][lane] = my_dot;
      __syncthreads();
      if (sub == 0 && lane < K)
        for (int i = 1; i < WPT; ++i) my_dot += part[wave + i][lane];
      __syncthreads();
    }
    if (t < T && sub == 0 && lane < K && (y_perm || my_p < 0)) dtopk_w[t * K + lane] = my_dot;
  }
}

// 64 columns per workgroup, chunks over its 16 wavefronts.
constexpr int kReduceWaves = 16;
__global__ void __launch_bounds__(kReduceWaves * kWave)
null_vector_reduce_kernel(const float* __restrict__ part, int64_t chunks, int d, float* __restrict__ dnull) {
  __shared__ double sum[kReduceWaves][kWave];
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int64_t c = (int64_t)blockIdx.x * kWave + lane;
  double s = 0.0;
  if (c < d) {
#pragma unroll 8
    for (int64_t i = wave; i < chunks; i += kReduceWaves) s += part[i * d + c];
  }
  sum[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && c < d) {
    for (int i = 1; i < kReduceWaves; ++i) s += sum[i][lane];
    dnull[c] = (float)s;
  }
}

template <typename RT, typename AT, typename ET, bool WEIGHTED>
hipError_t slot_sum(const SlotSumArgs& a, hipStream_t stream) {
  const int spans = (a.d + kSpan - 1) / kSpan;
  const int64_t blocks = std::min<int64_t>((a.T * spans + 3) / 4, 1 << 20);
  slot_sum_kernel<RT, AT, ET, WEIGHTED><<<(unsigned)blocks, kThreads, 0, stream>>>(
      static_cast<const RT*>(a.rows), a.slot_pos, a.topk_w, static_cast<const AT*>(a.shared),
      static_cast<const ET*>(a.null_src), a.null_stride, static_cast<ET*>(a.y), a.T, a.K, a.d, a.max_rows, spans);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_combine_rows(const SlotSumArgs& a, hipStream_t stream) {
  if (a.T <= 0) return hipSuccess;
  return with_rows(a.rows_dtype, [&](auto* r) {
    typedef std::remove_pointer_t<decltype(r)> RT;
    return a.out_dtype == MOE_BF16 ? slot_sum<RT, RT, bf16_t, true>(a, stream)
                                   : slot_sum<RT, RT, float, true>(a, stream);
  });
}

hipError_t launch_permute_bwd(const SlotSumArgs& a, hipStream_t stream) {
  if (a.T <= 0) return hipSuccess;
  return with_rows(a.rows_dtype, [&](auto* r) {
    return with_rows(a.out_dtype, [&](auto* e) {
      return slot_sum<std::remove_pointer_t<decltype(r)>, float, std::remove_pointer_t<decltype(e)>, false>(a, stream);
    });
  });
}

size_t combine_bwd_ws_bytes(int64_t T, int d, int null_kind) {
  return null_kind == MOE_NULL_CONSTANT ? (size_t)((T + kNullChunk - 1) / kNullChunk) * d * sizeof(float) : 0;
}

hipError_t launch_combine_bwd(const CombineBwdArgs& a, hipStream_t stream) {
  if (a.T <= 0) return hipSuccess;
  auto typed = [&](auto* r, auto* e) {
    typedef std::remove_pointer_t<decltype(r)> RT;
    typedef std::remove_pointer_t<decltype(e)> ET;
    float* dnull = a.null_stride ? a.dnull : nullptr;  // per token (copy)
    const bool vector = a.dnull && !a.null_stride;     // one vector (constant)
    const int64_t chunks = (a.T + kNullChunk - 1) / kNullChunk;
    const int spans = (a.d + kWave * kNullCols - 1) / (kWave * kNullCols);
    const unsigned extra = vector ? (unsigned)std::min<int64_t>((chunks * spans + 3) / 4, 1 << 20) : 0;
    auto go = [&](auto wpt) {
      constexpr int WPT = decltype(wpt)::value, kTokens = kThreads / kWave / WPT;
      const unsigned blocks = (unsigned)std::min<int64_t>((a.T + kTokens - 1) / kTokens, 1 << 20);
      combine_bwd_kernel<RT, ET, WPT><<<blocks + extra, kThreads, 0, stream>>>(
          static_cast<const ET*>(a.dy), static_cast<const RT*>(a.y_perm), a.slot_pos, a.topk_w,
          static_cast<const ET*>(a.null_src), a.null_stride, static_cast<RT*>(a.dy_perm), a.w_perm, a.row_slot,
          a.dtopk_w, dnull, a.T, a.K, a.d, a.max_rows, blocks, a.part);
    };
    // wavefronts per token by the spans of a row (bf16, 8 slots a quarter real, us with one,
    // two and four: 16384 x 512 16.4, 19.9 and 28.6; x 1024 37.1, 36.4 and 46.5; x 2048
    // 75.4, 69.9 and 66.7; 1000 x 4096 18.6, 11.8 and 9.5)
    if (a.d <= kSpan) go(std::integral_constant<int, 1>{});
    else if (a.d <= 2 * kSpan) go(std::integral_constant<int, 2>{});
    else go(std::integral_constant<int, 4>{});
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess || !vector) return err;
    null_vector_reduce_kernel<<<(unsigned)((a.d + kWave - 1) / kWave), kReduceWaves * kWave, 0, stream>>>(
        a.part, chunks, a.d, a.dnull);
    return hipGetLastError();
  };
  return with_rows(a.rows_dtype, [&](auto* r) {
    return a.bf16 ? typed(r, static_cast<bf16_t*>(nullptr)) : typed(r, static_cast<float*>(nullptr));
  });
}

}  // namespace moe
