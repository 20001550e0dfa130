// Products of rows in expert order with their expert's weights, over segments of any
// length (the grouped GEMM of the paper review "Improving MoE Compute Efficiency by
// Composing Weight and Data Sparsity", section 3 "implementation", as plain products with
// gradients, for experts of one's own):
//   product          out[p] = W[e] a[src(p)]           reduces over k_dim
//   data gradient    da[p] = W[e]^T dy[p]              reduces over n_out
//   weight gradient  dW[e] = add[e] + sum_p dy[p] a[src(p)]^T   reduces over the rows of e
// and the product with 4-bit weights (weights4.hpp), plain or as silu(W0 a) * (W1 a).
#include <algorithm>

#include "grouped_mm.hpp"
#include "rows.hpp"
#include "weights4.hpp"

namespace moe {

namespace {

__device__ __forceinline__ float load_any(int dtype, const void* p, int64_t i) {
  if (dtype == MOE_F32) return static_cast<const float*>(p)[i];
  if (dtype == MOE_BF16) return bf16_to_f32(static_cast<const bf16_t*>(p)[i]);
  return (float)static_cast<const half_t*>(p)[i];
}
__device__ __forceinline__ void store_any(int dtype, void* p, int64_t i, float v) {
  if (dtype == MOE_F32) static_cast<float*>(p)[i] = v;
  else if (dtype == MOE_BF16) static_cast<bf16_t*>(p)[i] = f32_to_bf16(v);
  else static_cast<half_t*>(p)[i] = (half_t)v;
}

// Tiles of 64 x 64 outputs, 4 x 4 a thread, 16 of the reduction at a time through LDS in
// float32: any type, any form.
constexpr int kT = 64, kTK = 16;

template <int FORM>
__global__ void __launch_bounds__(256) grouped_mm_kernel(GroupedMm g) {
  __shared__ Segments sg;
  __shared__ float L[kTK][kT + 4], R0[kTK][kT + 4], R1[kTK][kT + 4];
  const int I = FORM == kMmWgrad ? g.n_out : 0, J = FORM == kMmDgrad || FORM == kMmWgrad ? g.k_dim : g.n_out;
  const int nt = (J + kT - 1) / kT;
  const int total = build_segments(sg, g.offsets, g.groups, g.rows, kT, nt, I);
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  for (int t = blockIdx.x; t < total; t += gridDim.x) {
    const int e = segment_of(sg, g.groups, t);
    const int local = t - sg.prefix[e], start = sg.start[e], len = sg.len[e];
    const int mt = ((FORM == kMmWgrad ? I : len) + kT - 1) / kT;
    const int j0 = local / mt * kT, i0 = local % mt * kT;
    const int iend = FORM == kMmWgrad ? I : len;
    const int K = FORM == kMmWgrad ? len : FORM == kMmDgrad ? g.n_out : g.k_dim;
    auto source = [&](int p) -> int64_t {
      if (!g.a_rows) return p;
      return min<int64_t>(max<int64_t>(g.a_rows[p], 0), g.a_nrows - 1);
    };
    float acc[4][4] = {}, acc1[4][4] = {};
    for (int k0 = 0; k0 < K; k0 += kTK) {
      for (int x = threadIdx.x; x < kT * kTK; x += 256) {
        // neighbouring threads along the source's rows
        const int i = FORM == kMmWgrad ? x % kT : x / kTK, k = FORM == kMmWgrad ? x / kT : x % kTK;
        float l = 0.0f, r = 0.0f, r1 = 0.0f;
        if (k0 + k < K) {
          if (i0 + i < iend) {
            if (FORM == kMmWgrad) l = load_any(g.dtype, g.dy, (int64_t)(start + k0 + k) * g.ldy + i0 + i);
            else if (FORM == kMmDgrad) l = load_any(g.dtype, g.dy, (int64_t)(start + i0 + i) * g.ldy + k0 + k);
            else l = load_any(g.dtype, g.a, source(start + i0 + i) * g.lda + k0 + k);
          }
        }
        L[k][i] = l;
        const int j = FORM == kMmDgrad || FORM == kMmWgrad ? x % kT : x / kTK;
        const int kr = FORM == kMmDgrad || FORM == kMmWgrad ? x / kT : x % kTK;
        if (k0 + kr < K && j0 + j < J) {
          if (FORM == kMmWgrad) {
            r = load_any(g.dtype, g.a, source(start + k0 + kr) * g.lda + j0 + j);
          } else if (FORM == kMmDgrad) {
            r = load_any(g.dtype, g.w, ((int64_t)e * g.n_out + k0 + kr) * g.k_dim + j0 + j);
          } else {
            const int64_t at = ((int64_t)e * g.n_out + j0 + j) * g.k_dim + k0 + kr;
            if (FORM == kMm) r = load_any(g.dtype, g.w, at);
            else r = weight4(g.codes0, g.scales0, at);
            if (FORM == kMm4Swiglu) r1 = weight4(g.codes1, g.scales1, at);
          }
        }
        R0[kr][j] = r;
        if (FORM == kMm4Swiglu) R1[kr][j] = r1;
      }
      __syncthreads();
      for (int k = 0; k < kTK; ++k)
#pragma unroll
        for (int a = 0; a < 4; ++a)
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            acc[a][b] = fmaf(L[k][ty * 4 + a], R0[k][tx * 4 + b], acc[a][b]);
            if (FORM == kMm4Swiglu) acc1[a][b] = fmaf(L[k][ty * 4 + a], R1[k][tx * 4 + b], acc1[a][b]);
          }
      __syncthreads();
    }
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      const int i = i0 + ty * 4 + a;
      if (i >= iend) continue;
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int j = j0 + tx * 4 + b;
        if (j >= J) continue;
        float v = acc[a][b];
        if (FORM == kMm4Swiglu) v = silu(v) * acc1[a][b];
        int64_t at = (int64_t)(start + i) * g.ldo + j;
        if (FORM == kMmWgrad) {
          at = ((int64_t)e * g.n_out + i) * g.k_dim + j;
          if (g.add) v += g.add[at];
        }
        store_any(g.out_dtype, g.out, at, v);
      }
    }
  }
}

}  // namespace

hipError_t launch_grouped_mm(const GroupedMm& g, int num_cus, hipStream_t s) {
  if (g.form == kMm4 || g.form == kMm4Swiglu) return launch_grouped_mm_few(g, num_cus, s);
  if (g.dtype != MOE_F32) {
    // few rows: 73 us against 80 with 4 rows of each of 64 experts (n 2048, k 1536), 81 and 84
    // with 16, 111 and 87 with 32; 2 rows of two experts 8 and 18
    if (g.form == kMm && g.rows <= 16 * (int64_t)g.groups) return launch_grouped_mm_few(g, num_cus, s);
    return launch_grouped_mm16(g, num_cus, s);
  }
  const int I = g.form == kMmWgrad ? g.n_out : 0;
  const int J = g.form == kMmDgrad || g.form == kMmWgrad ? g.k_dim : g.n_out;
  const int64_t nt = (J + kT - 1) / kT;
  // no more tiles than this, whatever the offsets say: a segment ends in at most one partial tile
  const int64_t tiles = I ? (int64_t)g.groups * ((I + kT - 1) / kT) * nt : (g.rows / kT + g.groups) * nt;
  const unsigned blocks = (unsigned)std::min<int64_t>(tiles, 1 << 16);
  switch (g.form) {
    case kMm: grouped_mm_kernel<kMm><<<blocks, 256, 0, s>>>(g); break;
    case kMmDgrad: grouped_mm_kernel<kMmDgrad><<<blocks, 256, 0, s>>>(g); break;
    case kMmWgrad: grouped_mm_kernel<kMmWgrad><<<blocks, 256, 0, s>>>(g); break;
    case kMm4: grouped_mm_kernel<kMm4><<<blocks, 256, 0, s>>>(g); break;
    case kMm4Swiglu: grouped_mm_kernel<kMm4Swiglu><<<blocks, 256, 0, s>>>(g); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

}  // namespace moe
