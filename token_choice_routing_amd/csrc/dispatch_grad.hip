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
constexpr int kGroup = 4;  // slots whose rows are loaded before the first is added

// Position of a slot: a row of y_perm, or what stands in for one.
constexpr int kNullSlot = -1, kNoSlot = -2;

// y[t] = shared[t] + sum over slots of w r, in slot order (fmaf, one rounding). One
// wavefront per token and span of 64 E V columns; the token's positions and weights
// are read once by lanes 0..K-1 and broadcast. WEIGHTED false: every weight is 1.
template <typename RT, typename AT, typename ET, int E, int V, bool WEIGHTED>
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
    const int c0 = (int)(unit - t * spans) * (kWave * E * V) + lane * E;
    int my_p = kNoSlot;
    float my_w = 1.0f;
    if (lane < K) {
      my_p = slot_pos[t * K + lane];
      if (WEIGHTED) my_w = topk_w[t * K + lane];
      if (my_p == kNullSlot ? !null_src : (my_p < 0 || my_p >= max_rows)) my_p = kNoSlot;
    }
    float acc[V][E], nul[V][E];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = c0 + v * kWave * E;
#pragma unroll
      for (int j = 0; j < E; ++j) acc[v][j] = nul[v][j] = 0.0f;
      if (c < d) {
        if (shared) load_row<E>(shared + t * d + c, acc[v]);
        if (null_src) load_row<E>(null_src + t * null_stride + c, nul[v]);
      }
    }
    uint64_t todo = ballot(my_p != kNoSlot);
    while (todo) {
      int p[kGroup];
      float w[kGroup], r[kGroup][V][E];
#pragma unroll
      for (int g = 0; g < kGroup; ++g) {
        p[g] = kNoSlot;
        if (todo) {
          const int k = __builtin_ctzll(todo);
          todo &= todo - 1;
          p[g] = __builtin_amdgcn_readlane(my_p, k);
          w[g] = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(my_w), k));
          if (p[g] >= 0) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
              const int c = c0 + v * kWave * E;
              if (c < d) load_row<E>(rows + (int64_t)p[g] * d + c, r[g][v]);
            }
          }
        }
      }
#pragma unroll
      for (int g = 0; g < kGroup; ++g) {
        if (p[g] == kNoSlot) continue;
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
          for (int j = 0; j < E; ++j) {
            const float x = p[g] >= 0 ? r[g][v][j] : nul[v][j];
            acc[v][j] = WEIGHTED ? fmaf(w[g], x, acc[v][j]) : acc[v][j] + x;
          }
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = c0 + v * kWave * E;
      if (c < d) store_row<E>(y + t * d + c, acc[v]);
    }
  }
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, kWave);
  return v;
}

// The combine's gradient, one wavefront per token; V column vectors of E elements per
// lane and pass. ONE: the row fits one pass, so dy_t stays in registers over the slots.
template <typename RT, typename ET, int E, int V, bool ONE>
__global__ void __launch_bounds__(kThreads)
combine_bwd_kernel(const ET* __restrict__ dy, const RT* __restrict__ y_perm, const int32_t* __restrict__ slot_pos,
                   const float* __restrict__ topk_w, const ET* __restrict__ null_src, int64_t null_stride,
                   RT* __restrict__ dy_perm, float* __restrict__ w_perm, int32_t* __restrict__ row_slot,
                   float* __restrict__ dtopk_w, float* __restrict__ dnull, int64_t T, int K, int d,
                   int64_t max_rows) {
  const int lane = threadIdx.x & (kWave - 1);
  const int64_t nwaves = (int64_t)gridDim.x * (kThreads / kWave);
  const int span = kWave * E * V;
  for (int64_t t = (int64_t)blockIdx.x * (kThreads / kWave) + threadIdx.x / kWave; t < T; t += nwaves) {
    int my_p = kNoSlot;
    float my_w = 0.0f;
    if (lane < K) {
      my_p = slot_pos[t * K + lane];
      my_w = topk_w[t * K + lane];
      if (my_p != kNullSlot && (my_p < 0 || my_p >= max_rows)) my_p = kNoSlot;
      if (my_p >= 0) {
        if (w_perm) w_perm[my_p] = my_w;
        if (row_slot) row_slot[my_p] = (int32_t)(t * K + lane);
      }
    }
    float my_dot = 0.0f;  // lane k: the weight gradient of slot k
    const uint64_t nulls = ballot(my_p == kNullSlot);
    const ET* dyt = dy + t * d;
    float g[V][E];
    auto load_dy = [&](int c0) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = c0 + v * kWave * E + lane * E;
#pragma unroll
        for (int j = 0; j < E; ++j) g[v][j] = 0.0f;
        if (c < d) load_row<E>(dyt + c, g[v]);
      }
    };
    if (ONE) load_dy(0);
    // the expert rows, kGroup slots at a time
    uint64_t todo = ballot(my_p >= 0);
    while (todo && (dy_perm || (y_perm && dtopk_w))) {
      int p[kGroup], k[kGroup];
      float w[kGroup], dot[kGroup];
#pragma unroll
      for (int i = 0; i < kGroup; ++i) {
        p[i] = kNoSlot;
        k[i] = 0;
        w[i] = dot[i] = 0.0f;
        if (todo) {
          k[i] = __builtin_ctzll(todo);
          todo &= todo - 1;
          p[i] = __builtin_amdgcn_readlane(my_p, k[i]);
          w[i] = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(my_w), k[i]));
        }
      }
      for (int c0 = 0; c0 < d; c0 += span) {
        if (!ONE) load_dy(c0);
#pragma unroll
        for (int i = 0; i < kGroup; ++i) {
          if (p[i] < 0) continue;
#pragma unroll
          for (int v = 0; v < V; ++v) {
            const int c = c0 + v * kWave * E + lane * E;
            if (c >= d) continue;
            if (y_perm && dtopk_w) {
              float r[E];
              load_row<E>(y_perm + (int64_t)p[i] * d + c, r);
#pragma unroll
              for (int j = 0; j < E; ++j) dot[i] = fmaf(g[v][j], r[j], dot[i]);
            }
            if (dy_perm) {
              float o[E];
#pragma unroll
              for (int j = 0; j < E; ++j) o[j] = w[i] * g[v][j];
              store_row<E>(dy_perm + (int64_t)p[i] * d + c, o);
            }
          }
        }
      }
#pragma unroll
      for (int i = 0; i < kGroup; ++i) {
        const float s = wave_sum(dot[i]);
        if (p[i] >= 0 && lane == k[i]) my_dot = s;
      }
    }
    // the null slots: one product <dy_t, null source> for all of them, and the copied
    // token's gradient (sum of their weights) dy_t
    if (null_src && nulls && (dtopk_w || dnull)) {
      float wn = 0.0f;
      for (uint64_t m = nulls; m; m &= m - 1)
        wn += __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(my_w), __builtin_ctzll(m)));
      float dot = 0.0f;
      for (int c0 = 0; c0 < d; c0 += span) {
        if (!ONE) load_dy(c0);
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const int c = c0 + v * kWave * E + lane * E;
          if (c >= d) continue;
          if (dtopk_w) {
            float r[E];
            load_row<E>(null_src + t * null_stride + c, r);
#pragma unroll
            for (int j = 0; j < E; ++j) dot = fmaf(g[v][j], r[j], dot);
          }
          if (dnull) {
            float o[E];
#pragma unroll
            for (int j = 0; j < E; ++j) o[j] = wn * g[v][j];
            store_row<E>(dnull + t * d + c, o);
          }
        }
      }
      dot = wave_sum(dot);
      if (my_p == kNullSlot) my_dot = dot;
    } else if (dnull) {  // no null slot: the copied token gets nothing
      for (int c = lane * E; c < d; c += kWave * E) {
        float o[E];
#pragma unroll
        for (int j = 0; j < E; ++j) o[j] = 0.0f;
        store_row<E>(dnull + t * d + c, o);
      }
    }
    if (dtopk_w && lane < K && (y_perm || my_p < 0)) dtopk_w[t * K + lane] = my_dot;
  }
}

// Gradient of the constant null expert's vector, sum over tokens of (sum of the null
// slots' weights) dy_t: float32 partial sums over chunks of kNullChunk tokens, then a
// float64 sum of the partials in chunk order.
constexpr int kNullChunk = 64;
template <typename ET>
__global__ void __launch_bounds__(kThreads)
null_vector_partial_kernel(const ET* __restrict__ dy, const int32_t* __restrict__ slot_pos,
                           const float* __restrict__ topk_w, int64_t T, int K, int d, int64_t chunks,
                           float* __restrict__ part) {
  __shared__ float wn[kNullChunk];
  __shared__ int has[kNullChunk];
  for (int64_t chunk = blockIdx.x; chunk < chunks; chunk += gridDim.x) {
    const int64_t t0 = chunk * kNullChunk;
    const int n = (int)min<int64_t>(kNullChunk, T - t0);
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kThreads) {
      float s = 0.0f;
      int any = 0;
      for (int k = 0; k < K; ++k)
        if (slot_pos[(t0 + i) * K + k] == kNullSlot) {
          s += topk_w[(t0 + i) * K + k];
          any = 1;
        }
      wn[i] = s;
      has[i] = any;
    }
    __syncthreads();
    for (int64_t c = ((int64_t)blockIdx.y * kThreads + threadIdx.x) * 4; c < d;
         c += (int64_t)gridDim.y * kThreads * 4) {
      float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      for (int i = 0; i < n; ++i) {
        if (!has[i]) continue;
        float g[4];
        load_row<4>(dy + (t0 + i) * d + c, g);
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[j] = fmaf(wn[i], g[j], acc[j]);
      }
      store_row<4>(part + chunk * d + c, acc);
    }
  }
}
__global__ void __launch_bounds__(kThreads)
null_vector_reduce_kernel(const float* __restrict__ part, int64_t chunks, int d, float* __restrict__ dnull) {
  const int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (c >= d) return;
  double s = 0.0;
  for (int64_t i = 0; i < chunks; ++i) s += part[i * d + c];
  dnull[c] = (float)s;
}

template <typename RT, typename AT, typename ET, bool WEIGHTED>
hipError_t slot_sum(const SlotSumArgs& a, hipStream_t stream) {
  constexpr int E = 8;
  const int vectors = (a.d + kWave * E - 1) / (kWave * E);  // of one wavefront, per row
  auto go = [&](auto v) {
    constexpr int V = decltype(v)::value;
    const int spans = (vectors + V - 1) / V;
    const int64_t blocks = std::min<int64_t>((a.T * spans + 3) / 4, 1 << 20);
    slot_sum_kernel<RT, AT, ET, E, V, WEIGHTED><<<(unsigned)blocks, kThreads, 0, stream>>>(
        static_cast<const RT*>(a.rows), a.slot_pos, a.topk_w, static_cast<const AT*>(a.shared),
        static_cast<const ET*>(a.null_src), a.null_stride, static_cast<ET*>(a.y), a.T, a.K, a.d, a.max_rows, spans);
    return hipGetLastError();
  };
  return go(std::integral_constant<int, 2>{});
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
    constexpr int E = 8;
    const unsigned blocks = (unsigned)std::min<int64_t>((a.T + 3) / 4, 1 << 20);
    float* dnull = a.null_stride ? a.dnull : nullptr;  // per token; the constant's follows
    auto go = [&](auto kernel) {
      kernel<<<blocks, kThreads, 0, stream>>>(
          static_cast<const ET*>(a.dy), static_cast<const RT*>(a.y_perm), a.slot_pos, a.topk_w,
          static_cast<const ET*>(a.null_src), a.null_stride, static_cast<RT*>(a.dy_perm), a.w_perm, a.row_slot,
          a.dtopk_w, dnull, a.T, a.K, a.d, a.max_rows);
    };
    if (a.d <= 2 * kWave * E) go(combine_bwd_kernel<RT, ET, E, 2, true>);
    else if (a.d <= 4 * kWave * E) go(combine_bwd_kernel<RT, ET, E, 4, true>);
    else go(combine_bwd_kernel<RT, ET, E, 4, false>);
    hipError_t err = hipGetLastError();
    if (err != hipSuccess || !a.dnull || a.null_stride) return err;
    const int64_t chunks = (a.T + kNullChunk - 1) / kNullChunk;
    const dim3 grid((unsigned)std::min<int64_t>(chunks, 1 << 16),
                    (unsigned)std::min<int64_t>(((int64_t)a.d + 4 * kThreads - 1) / (4 * kThreads), 64));
    null_vector_partial_kernel<ET><<<grid, kThreads, 0, stream>>>(static_cast<const ET*>(a.dy), a.slot_pos, a.topk_w,
                                                                  a.T, a.K, a.d, chunks, a.part);
    if ((err = hipGetLastError()) != hipSuccess) return err;
    null_vector_reduce_kernel<<<(unsigned)((a.d + kThreads - 1) / kThreads), kThreads, 0, stream>>>(a.part, chunks,
                                                                                                  a.d, a.dnull);
    return hipGetLastError();
  };
  return with_rows(a.rows_dtype, [&](auto* r) {
    return a.bf16 ? typed(r, static_cast<bf16_t*>(nullptr)) : typed(r, static_cast<float*>(nullptr));
  });
}

}  // namespace moe
