// segments.cuh - the experts' token segments of a grouped call, as each CTA derives them from
// the offsets.
#pragma once

#include <cstdint>

#include "device.cuh"
#include "mxfp8.h"

namespace mxfp8 {

constexpr int kMaxExperts = 1024;  // scanned in shared memory

// Expert segmentation of the token rows for grouped calls. Every CTA re-derives the
// prefix sums of ceil(count / 128) from the offsets, so that no table has to be kept in
// global memory; invalid offsets make every CTA return without writing anything.
struct Segments {
  int32_t off[kMaxExperts + 1];
  int32_t tile_base[kMaxExperts + 1];  // prefix sum of ceil(count_e / 128)
  int32_t warp_sum[32];                // scratch of the block-wide scan
  int ok;
};

// The same in shared memory sized by the number of experts, for kernels whose loads need the L1
// cache that a table of kMaxExperts would take.
struct SegmentView {
  int32_t* off;
  int32_t* tile_base;
  int32_t* warp_sum;
  int& ok;
  static constexpr int words(int E) { return 2 * (E + 1) + 33; }
  __device__ SegmentView(int32_t* at, int E)
      : off(at), tile_base(at + E + 1), warp_sum(at + 2 * (E + 1)),
        ok(*reinterpret_cast<int*>(at + 2 * (E + 1) + 32)) {}
};

// The prefix sums come from a block-wide scan: each thread sums the tile counts of
// kMaxExperts / kThreads consecutive experts, a warp shuffle scan and the warps' totals
// place each thread's run, and the thread writes its experts' bases. A grouped launch runs
// this in every CTA, so a serial loop over the experts by one thread would cost each CTA
// microseconds.
template <int kThreads, typename S>
__device__ void load_segments(S& s, const int32_t* __restrict__ offsets, int E,
                              int64_t total_rows, int* status) {
  constexpr int kPer = kMaxExperts / kThreads;  // experts per thread
  static_assert(kPer * kThreads == kMaxExperts, "experts must split evenly over the CTA");
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  if (t == 0) s.ok = 1;
  __syncthreads();
  for (int i = t; i <= E; i += kThreads) s.off[i] = offsets[i];
  __syncthreads();
  int32_t tiles[kPer];
  int32_t mine = 0;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int e = t * kPer + j;
    int32_t n = 0;
    if (e < E) {
      const int32_t lo = s.off[e], hi = s.off[e + 1];
      if (hi < lo || (lo & 31) || (hi & 31)) s.ok = 0;
      n = hi > lo ? (hi - lo + 127) / 128 : 0;
    }
    tiles[j] = n;
    mine += n;
  }
  if (t == 0 && (s.off[0] != 0 || static_cast<int64_t>(s.off[E]) != total_rows)) s.ok = 0;
  int32_t incl = mine;  // inclusive scan within the warp
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int32_t v = __shfl_up_sync(0xFFFFFFFFu, incl, d);
    if (lane >= d) incl += v;
  }
  if (lane == 31) s.warp_sum[warp] = incl;
  __syncthreads();
  int32_t base = incl - mine;
  for (int w = 0; w < warp; ++w) base += s.warp_sum[w];
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int e = t * kPer + j;
    if (e < E) s.tile_base[e] = base;
    base += tiles[j];
  }
  if (t == kThreads - 1) s.tile_base[E] = base;  // the total: threads past E add nothing
  __syncthreads();
  if (t == 0 && !s.ok) latch_error(status, MXFP8_ERR_BAD_OFFSETS);
}

// Finds the expert owning global tile-row `t` (tile_base[e] <= t < tile_base[e+1]).
template <typename S>
__device__ __forceinline__ int find_expert(const S& s, int E, int t) {
  int lo = 0, hi = E - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (s.tile_base[mid] <= t) lo = mid; else hi = mid - 1;
  }
  return lo;
}

}  // namespace mxfp8
