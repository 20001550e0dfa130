// Segments of a grouped product: which rows each group owns and which tile a workgroup
// takes, from the offsets on the device.
#pragma once
#include "common.hpp"
#include "kernels.hpp"

namespace moe {

constexpr int kMmGroups = MOE_MAX_EXPERTS;
static_assert((kMmGroups + 1) % kWave == 0, "segment_of reads whole wavefronts of the table");

// Work of a weight gradient's tile beside its rows, in rows: its stores (256 KB of float32 take
// about as long as the products of 256 rows).
constexpr int kTileCost = 256;

// Row ranges of the groups and the running count of their output tiles.
struct Segments {
  int start[kMmGroups + 1];
  int len[kMmGroups + 1];
  int prefix[kMmGroups + 1];  // tiles before group e
  // weight gradient:
  int64_t cost[kMmGroups + 1];  // work before group e
  int order[kMmGroups + 1];     // largest_first(): the group at a place of the order,
  int skip[kMmGroups + 1];      // its tiles before the share,
  int count[kMmGroups + 1];     // and those in it
};

// Group e's rows are [a, b) with a = clamp(offsets[e], 0, rows), b = clamp(offsets[e + 1], a,
// rows): inside the buffers whatever the offsets hold. A group has ceil(extent / bm) * nt
// tiles, extent being its rows, or `fixed` where that is positive (a weight gradient: every
// group's output has n_out rows). Called by the whole workgroup (at least one wavefront);
// returns the number of tiles. `fixed` also fills in the work: a tile's is its group's rows and
// kTileCost more.
__device__ __forceinline__ int build_segments(Segments& sg, const int32_t* offsets, int groups, int64_t rows, int bm,
                                              int nt, int fixed) {
  if (threadIdx.x < kWave) {
    const int lane = threadIdx.x;
    constexpr int kPer = (kMmGroups + 1) / kWave;
    int32_t off[kPer + 1];  // all loads first
#pragma unroll
    for (int q = 0; q <= kPer; ++q) off[q] = offsets ? offsets[min(lane * kPer + q, groups)] : 0;
    int cnt[kPer], local = 0;
    int64_t work[kPer], lwork = 0;
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      const int e = lane * kPer + q;
      int a = 0, len = 0;
      if (e < groups) {
        len = (int)rows;
        if (offsets) {
          a = min(max(off[q], 0), (int)rows);
          len = min(max(off[q + 1], a), (int)rows) - a;
        }
      }
      sg.start[e] = a;
      sg.len[e] = len;
      cnt[q] = e < groups ? ((fixed > 0 ? fixed : len) + bm - 1) / bm * nt : 0;
      local += cnt[q];
      work[q] = (int64_t)cnt[q] * (len + kTileCost);
      lwork += work[q];
    }
    int incl = local;
    int64_t iwork = lwork;
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) {
      const int v = __shfl_up(incl, o, kWave);
      if (lane >= o) incl += v;
      if (fixed > 0) {
        const int64_t x = __shfl_up(iwork, o, kWave);
        if (lane >= o) iwork += x;
      }
    }
    int run = incl - local;
    iwork -= lwork;
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      sg.prefix[lane * kPer + q] = run;
      run += cnt[q];
      if (fixed > 0) sg.cost[lane * kPer + q] = iwork;
      iwork += work[q];
    }
  }
  __syncthreads();
  return sg.prefix[groups];
}

// The group of tile t (prefix[e] <= t < prefix[e + 1]), by every lane of a wavefront: its
// lanes count the groups that begin at or before t (as many as MOE_MAX_EXPERTS in four steps;
// a binary search's eight dependent LDS reads took 0.4 us a tile).
__device__ __forceinline__ int segment_of(const Segments& sg, int groups, int t) {
  const int lane = threadIdx.x & (kWave - 1);
  int n = 0;
#pragma unroll
  for (int q = 0; q < (kMmGroups + 1) / kWave; ++q) {
    const int e = q * kWave + lane, p = sg.prefix[e];
    n += __popcll(ballot(e < groups && p <= t));
  }
  return n - 1;
}

// The first tile of share x of 8 of a weight gradient's work, by every lane of a wavefront: the
// groups' rows, and with them their tiles' times, differ much (64 experts of 18 to 3120 rows, 1536 x
// 2048: 403 us with equal numbers of tiles, 308 so).
__device__ __forceinline__ int work_share(const Segments& sg, int groups, int total, int x) {
  if (x >= 8) return total;
  const int lane = threadIdx.x & (kWave - 1);
  const int64_t at = sg.cost[groups] / 8 * x;
  int n = 0;
#pragma unroll
  for (int q = 0; q < (kMmGroups + 1) / kWave; ++q) {
    const int e = q * kWave + lane;
    const int64_t c = sg.cost[e];
    n += __popcll(ballot(e < groups && c <= at));
  }
  const int e = max(n - 1, 0);
  const int64_t within = (at - sg.cost[e]) / (sg.len[e] + kTileCost);
  return min(sg.prefix[e] + (int)within, total);
}

// Puts the groups of the tiles [first, last) of a weight gradient in order of their rows, most
// first, and the table's prefixes into that order (counted from 0): the workgroups of an XCD
// then take tiles of one group after the other's as before, but those that get one tile more
// of a group than others do so by turns among groups of like size, and the last tiles are the
// shortest (32768 rows of 64 experts as uneven as routing of skewed popularity makes them: 356 us
// without, 332 so). Called by the whole workgroup; last > first.
__device__ __forceinline__ void largest_first(Segments& sg, int groups, int first, int last) {
  const int lo = segment_of(sg, groups, first), m = segment_of(sg, groups, last - 1) - lo + 1;
  __syncthreads();  // every wavefront is done with the table as it was
  if (threadIdx.x < kWave) {
    const int lane = threadIdx.x;
    for (int i = lane; i <= kMmGroups; i += kWave) sg.count[i] = 0;
    for (int i = lane; i < m; i += kWave) {
      const int e = lo + i, len = sg.len[e];
      int rank = 0;
      for (int f = lo; f < lo + m; ++f) {
        const int l = sg.len[f];
        rank += l > len || (l == len && f < e);
      }
      const int from = max(sg.prefix[e], first);
      sg.order[rank] = e;
      sg.skip[rank] = from - sg.prefix[e];
      sg.count[rank] = min(sg.prefix[e + 1], last) - from;
    }
    constexpr int kPer = (kMmGroups + 1) / kWave;
    int cnt[kPer], local = 0;
#pragma unroll
    for (int q = 0; q < kPer; ++q) local += cnt[q] = sg.count[lane * kPer + q];
    int incl = local;
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) {
      const int v = __shfl_up(incl, o, kWave);
      if (lane >= o) incl += v;
    }
    int run = incl - local;
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      sg.prefix[lane * kPer + q] = run;
      run += cnt[q];
    }
  }
  __syncthreads();
}

}  // namespace moe
