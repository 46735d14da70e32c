// routing.cu - tokens sorted by expert, their rows copied into the experts' segments, and the
// experts' results summed back, with the gradients: what stands around the grouped quantizers
// and GEMMs of a mixture-of-experts layer.
//
// "End-to-End MXFP8 RL on Blackwell" (verl blog post) trains such a model (section "A held-out
// workload, and end to end", Table 4) with token segments padded to multiples of 32 (section
// "The pipeline", learner paragraph); it does not describe how the segments are made.
//
// Entry i = t top_k + j is token t's j-th choice, expert id_i. Entries keep their order within
// an expert, so the plan is the same in every run:
//   row_i = off[e] + #{i' < i : id_i' = e},  e = id_i;  off[e + 1] = off[e] + 32 ceil(count_e / 32)
//   dispatch   out[row_i]  = w_i x[t]
//   combine    out[t]      = sum_j w_i y[row_i]
//   gradients  dy[row_i]   = w_i dout[t],  dw_i = <dout[t], y[row_i]>
// Products and sums are FP32, each result is rounded once. Sums over a token's choices run in
// the order of j, sums over columns in an order that depends on the sizes alone.

#include <algorithm>
#include <atomic>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "device.cuh"
#include "internal.h"
#include "mxfp8.h"

namespace mxfp8 {
namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;

// ------------------------------------------------------------------------ sort by expert

constexpr int kRouteThreads = 1024, kRouteWarps = kRouteThreads / 32;
constexpr int kMaxExperts = 1024;   // one thread each
constexpr int kMaxRouteCtas = 16;   // of the cluster (more than 8 by leave)
constexpr int kBatch = 16;          // 32-entry groups that a warp keeps in registers
constexpr uint32_t kNoKey = 0xFFFFu;
static_assert(kMaxExperts <= kRouteThreads, "one thread an expert");

struct RouteParams {
  const int64_t* ids;
  int64_t n;            // entries
  int64_t per_warp;     // entries of a warp, a multiple of 32
  int E;
  int key_bits;         // of E - 1
  int64_t rows;
  int32_t* offsets;
  int32_t* row_of;
  int32_t* entry_of;
  int* status;
};

// Stable counting sort by one cluster of CTAs. Each warp owns a contiguous run of entries, 32 of
// them a group: the last lane of those with the same expert adds their number to the warp's own
// counter of that expert, and what stood there is the number of entries before the group. A thread
// per expert then turns the counters into places (over the warps of a CTA, then over the CTAs,
// whose totals go round through distributed shared memory), and the entries take them, in the
// order of their rows through shared memory: an SM stores to one line a clock, and scattered
// stores of 4 bytes took 4 us of 12 on 8 CTAs. Runs that do not fit the registers are read twice.
// One launch, no workspace, and nothing depends on timing: only one warp adds to a counter, group
// by group. Bound by the chain of these steps, each 0.3 to 1 us: 8 entries of 128 experts 3.2 us,
// 8192 4.8, 65536 8.5, 524288 39.
__global__ void __launch_bounds__(kRouteThreads) route_kernel(const RouteParams p) {
  extern __shared__ __align__(16) uint32_t dyn[];
  uint32_t* total = dyn;                                  // [CTAs][E], every CTA's
  uint32_t* count = dyn + ((gridDim.x * p.E + 3) & ~3u);  // [warps][E], and then:
  uint2* sorted = reinterpret_cast<uint2*>(count);        // rows and entries of the CTA, by row
  __shared__ uint32_t first_row[kMaxExperts];             // of this CTA's entries, by expert
  __shared__ uint32_t first_place[kMaxExperts];           // of them in `sorted`
  __shared__ uint2 warp_sum[kRouteWarps];
  __shared__ uint32_t all_rows, all_places;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, E = p.E;
  const int ctas = static_cast<int>(gridDim.x), rank = static_cast<int>(blockIdx.x);
  for (int i = tid; i < kRouteWarps * E; i += kRouteThreads) count[i] = 0;
  if (ctas > 1) cluster_arrive();   // this CTA has started: its shared memory may be written
  grid_dependency_wait();
  grid_launch_dependents();

  uint32_t* mine = count + warp * E;
  const int64_t begin = (static_cast<int64_t>(rank) * kRouteWarps + warp) * p.per_warp;
  const int64_t end = begin + p.per_warp < p.n ? begin + p.per_warp : p.n;
  // Of the lane's entry in each group: its expert (kNoKey for none) in the upper half, and what
  // its counter gave, at most 512, in the lower.
  uint32_t held[kBatch];
  bool bad = false;
  const auto read = [&](int64_t at) {
#pragma unroll
    for (int g = 0; g < kBatch; ++g) {
      if (at + 32 * g >= end) break;   // the same in all lanes
      const int64_t i = at + 32 * g + lane;
      const int64_t id = i < end ? p.ids[i] : -1;
      bad |= id >= E;
      held[g] = (id < 0 || id >= E ? kNoKey : static_cast<uint32_t>(id)) << 16;
    }
  };
  // Adds a group's keys to the warp's counters; returns the place of the lane's.
  const auto take = [&](uint32_t key) {
    // Lanes of the same key, from a vote on each of its bits (match.any takes longer the more keys
    // there are: 13.9 us of 8192 x 8 entries of 128 experts on 8 CTAs, 12.7 with votes).
    unsigned same = __ballot_sync(kFull, key != kNoKey);
    for (int b = 0; b < p.key_bits; ++b) {
      const bool set = key >> b & 1;
      const unsigned with = __ballot_sync(kFull, set);
      same &= set ? with : ~with;
    }
    if (key == kNoKey) same = 0;
    const int last = 31 - __clz(same | 1u);
    const uint32_t before = same ? mine[key] : 0u;
    __syncwarp();
    if (same && lane == last) mine[key] = before + __popc(same);
    __syncwarp();
    return before + __popc(same & ((1u << lane) - 1u));
  };
  const bool held_all = p.per_warp <= 32 * kBatch;
  if (begin < end) read(begin);
  __syncthreads();
  if (held_all) {
#pragma unroll
    for (int g = 0; g < kBatch; ++g) {
      if (begin + 32 * g >= end) break;
      held[g] += take(held[g] >> 16);
    }
  } else {   // only counted: the order comes with the second reading
    for (int64_t at = begin; at < end; at += 32 * kBatch) {
      if (at != begin) read(at);
#pragma unroll
      for (int g = 0; g < kBatch; ++g) {
        if (at + 32 * g >= end) break;
        if (held[g] >> 16 != kNoKey) atomicAdd(mine + (held[g] >> 16), 1u);
      }
    }
  }
  if (bad) latch_error(p.status, MXFP8_ERR_BAD_EXPERT);
  __syncthreads();

  // counters to places among the CTA's entries of that expert
  uint32_t sum = 0;
  if (tid < E) {
#pragma unroll 8
    for (int w = 0; w < kRouteWarps; ++w) {
      const uint32_t c = count[w * E + tid];
      count[w * E + tid] = sum;
      sum += c;
    }
    total[rank * E + tid] = sum;
  }
  if (ctas > 1) {
    cluster_wait();
    if (tid < E)
      for (int c = 0; c < ctas; ++c)
        if (c != rank)
          st_cluster_u32(cluster_map(&total[rank * E + tid], static_cast<uint32_t>(c)), sum);
    cluster_sync();
  }

  // Scans over the experts: of their counts rounded up to 32, the segments, and of this CTA's
  // counts.
  uint32_t before = 0, all = 0;
  if (tid < E)
    for (int c = 0; c < ctas; ++c) {
      const uint32_t v = total[c * E + tid];
      before += c < rank ? v : 0;
      all += v;
    }
  const uint32_t padded = (all + 31u) & ~31u;
  uint2 incl = make_uint2(padded, sum);
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t x = __shfl_up_sync(kFull, incl.x, d), y = __shfl_up_sync(kFull, incl.y, d);
    if (lane >= d) incl = make_uint2(incl.x + x, incl.y + y);
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  uint2 base = make_uint2(incl.x - padded, incl.y - sum);
  if (tid < E) {
    for (int w = 0; w < warp; ++w) {
      base.x += warp_sum[w].x;
      base.y += warp_sum[w].y;
    }
    first_row[tid] = base.x + before;
    first_place[tid] = base.y;
    // of the whole expert, for the padding below: the end of its entries
    total[tid] = base.x + all;
    if (tid == E - 1) {
      all_rows = base.x + padded;
      all_places = base.y + sum;
    }
  }
  __syncthreads();
  const bool fits = all_rows <= p.rows;   // n + 31 E is below 2^32: nothing wrapped
  if (rank == 0) {
    if (tid < E) p.offsets[tid] = fits ? static_cast<int32_t>(base.x) : 0;
    if (tid == 0) {
      p.offsets[E] = static_cast<int32_t>(p.rows);
      if (!fits) latch_error(p.status, MXFP8_ERR_BAD_OFFSETS);
    }
  }
  const int64_t step = static_cast<int64_t>(ctas) * kRouteThreads;
  const int64_t thread = static_cast<int64_t>(rank) * kRouteThreads + tid;
  if (!fits) {   // a plan without entries: valid offsets, padding everywhere
    for (int64_t i = thread; i < p.n; i += step) p.row_of[i] = -1;
    for (int64_t r = thread; r < p.rows; r += step) p.entry_of[r] = -1;
    return;
  }

  if (held_all) {
#pragma unroll
    for (int g = 0; g < kBatch; ++g) {   // places among the CTA's, at most 16384
      if (begin + 32 * g >= end) break;
      if (held[g] >> 16 != kNoKey) held[g] += mine[held[g] >> 16];
    }
    __syncthreads();   // the counters have been read: `sorted` takes their place
#pragma unroll
    for (int g = 0; g < kBatch; ++g) {
      if (begin + 32 * g >= end) break;
      const int64_t i = begin + 32 * g + lane;
      const uint32_t key = held[g] >> 16, place = held[g] & 0xFFFFu;
      int32_t row = -1;
      if (key != kNoKey) {
        row = static_cast<int32_t>(first_row[key] + place);
        sorted[first_place[key] + place] =
            make_uint2(static_cast<uint32_t>(row), static_cast<uint32_t>(i));
      }
      if (i < end) p.row_of[i] = row;
    }
    __syncthreads();
    for (uint32_t at = tid; at < all_places; at += kRouteThreads)
      p.entry_of[sorted[at].x] = static_cast<int32_t>(sorted[at].y);
  } else {
    for (int64_t at = begin; at < end; at += 32 * kBatch) {
      read(at);
#pragma unroll
      for (int g = 0; g < kBatch; ++g) {
        if (at + 32 * g >= end) break;
        const int64_t i = at + 32 * g + lane;
        const uint32_t key = held[g] >> 16, place = take(key);   // on from the warp's first places
        int32_t row = -1;
        if (key != kNoKey) {
          row = static_cast<int32_t>(first_row[key] + place);
          p.entry_of[row] = static_cast<int32_t>(i);
        }
        if (i < end) p.row_of[i] = row;
      }
    }
  }
  // rows of no entry: the ends of the segments, and all that is left after the last
  for (int e = rank * kRouteWarps + warp; e < E; e += ctas * kRouteWarps) {
    const uint32_t r = total[e] + static_cast<uint32_t>(lane);
    if (r < ((total[e] + 31u) & ~31u)) p.entry_of[r] = -1;
  }
  for (int64_t r = static_cast<int64_t>(all_rows) + thread; r < p.rows; r += step)
    p.entry_of[r] = -1;
}

// ------------------------------------------------------------------ values of a row

// V consecutive elements of a row, moved as one access of kBytes and computed with in FP32.
template <int kBytes>
struct Raw;
template <>
struct Raw<16> { using type = uint4; };
template <>
struct Raw<8> { using type = uint2; };
template <>
struct Raw<4> { using type = uint32_t; };
template <>
struct Raw<2> { using type = uint16_t; };

template <typename T, int V>
struct Pack {
  using raw = typename Raw<V * static_cast<int>(sizeof(T))>::type;
};

__device__ __forceinline__ uint4 load_once(const uint4* p) { return ld_nc_v4(p); }
__device__ __forceinline__ uint2 load_once(const uint2* p) { return __ldg(p); }
__device__ __forceinline__ uint32_t load_once(const uint32_t* p) { return __ldg(p); }
__device__ __forceinline__ uint16_t load_once(const uint16_t* p) { return __ldg(p); }

// The same of memory that the kernel itself may overwrite (a result in place of what it is made
// from): an ordinary load, since a non-coherent one need not stay before the store.
template <bool kMayBeWritten, typename R>
__device__ __forceinline__ R load_operand(const R* p) {
  if constexpr (kMayBeWritten) return *p;
  return load_once(p);
}

__device__ __forceinline__ void zero(uint4& v) { v = make_uint4(0, 0, 0, 0); }
__device__ __forceinline__ void zero(uint2& v) { v = make_uint2(0, 0); }
__device__ __forceinline__ void zero(uint32_t& v) { v = 0; }
__device__ __forceinline__ void zero(uint16_t& v) { v = 0; }

template <typename T, int V>
__device__ __forceinline__ void unpack(const typename Pack<T, V>::raw& r, float (&x)[V]) {
  if constexpr (sizeof(r) == 2) {
    x[0] = __uint_as_float(static_cast<uint32_t>(r) << 16);
  } else {
    uint32_t w[sizeof(r) / 4];
    memcpy(w, &r, sizeof(r));
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(r) / 4); ++i) {
      if constexpr (sizeof(T) == 4) {
        x[i] = __uint_as_float(w[i]);
      } else {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    }
  }
}

template <typename T, int V>
__device__ __forceinline__ typename Pack<T, V>::raw pack(const float (&x)[V]) {
  typename Pack<T, V>::raw r;
  if constexpr (sizeof(r) == 2) {
    r = static_cast<uint16_t>(cvt_bf16x2(0.f, x[0]));
  } else {
    uint32_t w[sizeof(r) / 4];
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(r) / 4); ++i)
      w[i] = sizeof(T) == 4 ? __float_as_uint(x[i])
                            : cvt_bf16x2(x[(2 * i + 1) % V], x[(2 * i) % V]);
    memcpy(&r, w, sizeof(r));
  }
  return r;
}

struct RowsParams {
  const void* src;         // dispatch: x; combine: y; gradient: dout
  const void* y;           // gradient
  const float* weights;    // [tokens][k], or nullptr
  const int32_t* row_of;   // [tokens][k]
  const int32_t* entry_of; // [rows]
  int64_t tokens, cols, rows;
  int k;
  void* out;
  float* grad_w;           // gradient
  int* status;
};

// Rows without an entry, set to zero: a warp looks at every (warps of the grid)-th row, so that a
// run of them, as the last segment takes it, is spread over the SMs.
template <typename T, int V>
__device__ __forceinline__ void zero_padding(const RowsParams& p, int64_t cta, int64_t ctas,
                                             int warps) {
  using raw = typename Pack<T, V>::raw;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  raw none;
  zero(none);
  const int64_t vecs = p.cols / V, step = ctas * warps;
  for (int64_t r0 = warp * ctas + cta; r0 < p.rows; r0 += 32 * step) {
    const int64_t mine = r0 + lane * step;   // the row that the lane looks at
    unsigned pad = __ballot_sync(kFull, mine < p.rows && p.entry_of[mine] < 0);
    for (; pad; pad &= pad - 1) {
      raw* out = reinterpret_cast<raw*>(p.out) + (r0 + (__ffs(pad) - 1) * step) * vecs;
      for (int64_t c = lane; c < vecs; c += 32) out[c] = none;
    }
  }
}

// A row of the plan as the kernels use it: -1 where there is none. One past the rows (a plan
// of other sizes) is latched, and skipped.
__device__ __forceinline__ int32_t plan_row(const RowsParams& p, int64_t entry) {
  const int32_t r = p.row_of[entry];
  if (r < p.rows) return r;
  latch_error(p.status, MXFP8_ERR_BAD_OFFSETS);
  return -1;
}

// ------------------------------------------------------------------------------ dispatch

constexpr int kThreads = 256, kWarps = kThreads / 32;

// Accesses of a lane: 64 bytes, or 16 of the smallest.
template <size_t kBytes>
constexpr int kDispatchU = kBytes >= 4 ? 64 / static_cast<int>(kBytes) : 16;

// A warp reads a piece of a token's row once and writes it to the token's k rows; the rows of
// no entry are zeroed on the side. Bound by the writes: 8192 tokens of 2048 BF16 columns, 8 experts
// each, 50 us (6.4 TB/s). Rows of less than 16-byte accesses start anywhere in a line: there the
// piece of each row is moved to the left so that stores start on lines, and x is read again, from
// L1, for each row. 8192 tokens of 1999 FP32 columns 106 us (129 with one reading and stores across
// lines), in BF16 74 (80); 1021 of them in FP32 with 6 experts each 12.6 (13.7).
template <typename T, int V, bool kWeighted>
__global__ void __launch_bounds__(kThreads) dispatch_kernel(const RowsParams p) {
  using raw = typename Pack<T, V>::raw;
  constexpr int kU = kDispatchU<sizeof(raw)>;
  constexpr bool kAligned = sizeof(raw) == 16;
  constexpr int kLine = 128 / static_cast<int>(sizeof(raw));
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  const int64_t vecs = p.cols / V;
  const int64_t c0 = static_cast<int64_t>(blockIdx.y) * 32 * kU + lane;
  if (t < p.tokens) {
    const raw* x = reinterpret_cast<const raw*>(p.src) + t * vecs;
    raw v[kU];
    const auto load = [&](int64_t c) {
#pragma unroll
      for (int u = 0; u < kU; ++u)
        if (c + 32 * u >= 0 && c + 32 * u < vecs) v[u] = load_once(x + c + 32 * u);
    };
    const auto weighed = [&](const raw& r, float w) {
      if constexpr (!kWeighted) return r;
      float f[V];
      unpack<T, V>(r, f);
#pragma unroll
      for (int i = 0; i < V; ++i) f[i] = __fmul_rn(f[i], w);
      return pack<T, V>(f);
    };
    if constexpr (kAligned) load(c0);
    for (int j0 = 0; j0 < p.k; j0 += 32) {
      const int left = p.k - j0 < 32 ? p.k - j0 : 32;
      int32_t my_row = -1;
      float my_w = 1.f;
      if (lane < left) {
        my_row = plan_row(p, t * p.k + j0 + lane);
        if (kWeighted && my_row >= 0) my_w = p.weights[t * p.k + j0 + lane];
      }
      for (int j = 0; j < left; ++j) {
        const int32_t r = __shfl_sync(kFull, my_row, j);
        const float w = kWeighted ? __shfl_sync(kFull, my_w, j) : 1.f;
        if (r < 0) continue;
        raw* out = reinterpret_cast<raw*>(p.out) + r * vecs;
        int64_t c = c0;
        if constexpr (!kAligned) {
          c -= (reinterpret_cast<uintptr_t>(out) / sizeof(raw)) % kLine;
          load(c);
        }
#pragma unroll
        for (int u = 0; u < kU; ++u)
          if (c + 32 * u >= 0 && c + 32 * u < vecs) out[c + 32 * u] = weighed(v[u], w);
        if constexpr (!kAligned)   // what the last piece leaves of the row
          if (blockIdx.y == gridDim.y - 1)
            for (int64_t i = c + 32 * kU; i < vecs; i += 32) out[i] = weighed(load_once(x + i), w);
      }
    }
  }
  const int64_t ctas = static_cast<int64_t>(gridDim.x) * gridDim.y;
  zero_padding<T, V>(p, static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x, ctas, kWarps);
}

// ------------------------------------------------------------------------------- combine

// A warp sums a piece (kC times 32 lanes x V columns) of a token's k rows, kU of them at a time:
// enough of both that a lane has 128 bytes on their way (64 in accesses of 2 bytes, 256 in those of 8).
// Bound by the reads: 8192 tokens of 2048 BF16 columns, 8 experts each, 46 us (6.5 TB/s); with 1999
// columns, 2-byte accesses, 67 (4.4).
template <typename T, int V, bool kWeighted, int kU, int kC>
__global__ void __launch_bounds__(kThreads) combine_kernel(const RowsParams p) {
  using raw = typename Pack<T, V>::raw;
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  const int64_t vecs = p.cols / V;
  const int64_t c0 = static_cast<int64_t>(blockIdx.y) * 32 * kC + lane;
  if (t >= p.tokens) return;
  const raw* y = reinterpret_cast<const raw*>(p.src) + c0;
  float sum[kC][V];
#pragma unroll
  for (int q = 0; q < kC; ++q)
#pragma unroll
    for (int i = 0; i < V; ++i) sum[q][i] = 0.f;
  for (int j0 = 0; j0 < p.k; j0 += 32) {
    const int left = p.k - j0 < 32 ? p.k - j0 : 32;
    int32_t my_row = -1;
    float my_w = 1.f;
    if (lane < left) {
      my_row = plan_row(p, t * p.k + j0 + lane);
      if (kWeighted && my_row >= 0) my_w = p.weights[t * p.k + j0 + lane];
    }
    for (int j = 0; j < left; j += kU) {
      raw v[kU][kC];
      int32_t r[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        r[u] = __shfl_sync(kFull, my_row, (j + u) & 31);
        if (j + u >= left) r[u] = -1;
#pragma unroll
        for (int q = 0; q < kC; ++q)
          if (r[u] >= 0 && c0 + 32 * q < vecs) v[u][q] = load_once(y + r[u] * vecs + 32 * q);
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const float w = kWeighted ? __shfl_sync(kFull, my_w, (j + u) & 31) : 1.f;
        if (r[u] < 0) continue;
#pragma unroll
        for (int q = 0; q < kC; ++q) {
          if (c0 + 32 * q >= vecs) continue;
          float f[V];
          unpack<T, V>(v[u][q], f);
#pragma unroll
          for (int i = 0; i < V; ++i)
            sum[q][i] = kWeighted ? fmaf(w, f[i], sum[q][i]) : sum[q][i] + f[i];
        }
      }
    }
  }
  raw* out = reinterpret_cast<raw*>(p.out) + t * vecs + c0;
#pragma unroll
  for (int q = 0; q < kC; ++q)
    if (c0 + 32 * q < vecs) out[32 * q] = pack<T, V>(sum[q]);
}

// -------------------------------------------------------------------- combine's gradient

constexpr int kGradThreads = 128;

// Sums of N values over the lanes of a warp; lane l < N gets the l-th (N a power of two).
template <int N>
__device__ __forceinline__ float sums_of(float (&x)[N], int lane) {
#pragma unroll
  for (int n = N, d = 16; n > 1; n /= 2, d /= 2) {
    // lanes whose bit d is set go on with the upper half of the values, the others with the lower
#pragma unroll
    for (int i = 0; i < n / 2; ++i) {
      const float send = lane & d ? x[i] : x[i + n / 2], keep = lane & d ? x[i + n / 2] : x[i];
      x[i] = keep + __shfl_xor_sync(kFull, send, d);
    }
  }
  float v = x[0];
#pragma unroll
  for (int d = 16 / N; d > 0; d /= 2) v += __shfl_xor_sync(kFull, v, d);
  // value i is in the lanes whose bits from 16 down spell i
  return __shfl_sync(kFull, v, (lane % N) * (32 / N));
}

// A group of kGroup threads (a warp, or the CTA) takes a token: it reads dout[t] and the token's
// rows of y, kU rows and kC times kGroup accesses of each at a time, writes w dout[t] to the rows'
// gradients and sums the products for the weights'. The sums are joined over the lanes, then over
// the warps in order. The rows' gradient may stand in y's place: a thread reads what it overwrites
// first. Bound by memory: 8192 tokens of 2048 BF16 columns, 8 experts each, 91 us (6.5 TB/s), in y's
// place 92, without the rows' gradient 44 (6.8); 509 tokens of 1033 FP32 columns, 4 each, a tenth of them
// dropped, 4.8 us (4.2 TB/s, of which 2 are the launch).
template <typename T, int V, int kGroup, bool kRows, int kU, int kC>
__global__ void __launch_bounds__(kGradThreads) combine_grad_kernel(const RowsParams p) {
  using raw = typename Pack<T, V>::raw;
  __shared__ float part[kGradThreads / 32][kU];
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int in_group = threadIdx.x % kGroup;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (kGradThreads / kGroup) +
                    threadIdx.x / kGroup;
  const int64_t vecs = p.cols / V;
  const raw* y = reinterpret_cast<const raw*>(p.y);
  raw* out = reinterpret_cast<raw*>(p.out);
  const bool live = t < p.tokens;
  const raw* g = reinterpret_cast<const raw*>(p.src) + (live ? t : 0) * vecs;
  for (int j0 = 0; j0 < p.k; j0 += kU) {
    int32_t r[kU];
    float w[kU], dot[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const bool there = live && j0 + u < p.k;
      r[u] = there ? plan_row(p, t * p.k + j0 + u) : -1;
      w[u] = r[u] >= 0 ? p.weights[t * p.k + j0 + u] : 0.f;
      dot[u] = 0.f;
    }
    if (live) {
      for (int64_t c0 = in_group; c0 < vecs; c0 += kGroup * kC) {
        raw gr[kC], v[kU][kC];
#pragma unroll
        for (int q = 0; q < kC; ++q)
          if (c0 + kGroup * q < vecs) gr[q] = load_once(g + c0 + kGroup * q);
#pragma unroll
        for (int u = 0; u < kU; ++u)
#pragma unroll
          for (int q = 0; q < kC; ++q)
            if (r[u] >= 0 && c0 + kGroup * q < vecs)
              v[u][q] = load_operand<kRows>(y + r[u] * vecs + c0 + kGroup * q);
#pragma unroll
        for (int q = 0; q < kC; ++q) {
          const int64_t c = c0 + kGroup * q;
          if (c >= vecs) continue;
          float gv[V];
          unpack<T, V>(gr[q], gv);
#pragma unroll
          for (int u = 0; u < kU; ++u) {
            if (r[u] < 0) continue;
            float f[V];
            unpack<T, V>(v[u][q], f);
#pragma unroll
            for (int i = 0; i < V; ++i) dot[u] = fmaf(gv[i], f[i], dot[u]);
            if constexpr (kRows) {
#pragma unroll
              for (int i = 0; i < V; ++i) f[i] = __fmul_rn(gv[i], w[u]);
              out[r[u] * vecs + c] = pack<T, V>(f);
            }
          }
        }
      }
    }
    const float sum = sums_of<kU>(dot, lane);
    if constexpr (kGroup == 32) {
      if (live && lane < kU && j0 + lane < p.k) p.grad_w[t * p.k + j0 + lane] = sum;
    } else {
      if (lane < kU) part[warp][lane] = sum;
      __syncthreads();
      if (live && threadIdx.x < kU && j0 + static_cast<int>(threadIdx.x) < p.k) {
        float all = 0.f;
#pragma unroll
        for (int q = 0; q < kGradThreads / 32; ++q) all += part[q][threadIdx.x];
        p.grad_w[t * p.k + j0 + threadIdx.x] = all;
      }
      __syncthreads();
    }
  }
  if constexpr (kRows)
    zero_padding<T, V>(p, blockIdx.x, gridDim.x, kGradThreads / 32);
}

template <typename... KArgs, typename... Args>
cudaError_t launch(void (*k)(KArgs...), dim3 grid, int threads, int cluster, size_t dyn,
                   cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.dynamicSmemBytes = dyn;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  cfg.attrs = attr;
  cfg.numAttrs = pdl_attr(&attr[0]);
  if (cluster > 1) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attr[cfg.numAttrs].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[cfg.numAttrs].val.clusterDim.y = 1;
    attr[cfg.numAttrs].val.clusterDim.z = 1;
    ++cfg.numAttrs;
  }
  return cudaLaunchKernelEx(&cfg, k, args...);
}

RowsParams rows_params(const RowsArgs& a) {
  return RowsParams{a.src, a.y, a.weights, a.row_of, a.entry_of, a.tokens, a.cols, a.rows, a.k,
                    a.out, a.grad_w, a.status};
}

// CTAs that the padding wants: a few tokens have much of it (8 of them with 64 experts each of
// 2048 columns: 17 us where the 8 tokens' CTAs alone write it). 8 warps an SM: 37 tokens with 8 of
// 128 experts 5.4 us, 300 tokens 6.3; with 32 warps 7.1 and 9.5.
int64_t padding_ctas(int64_t rows, int warps) {
  const int64_t most = int64_t{8} * num_sms() / warps, all = (rows + warps - 1) / warps;
  return all < most ? all : most;
}

template <typename T, int V>
cudaError_t launch_dispatch_v(const RowsArgs& a, cudaStream_t stream) {
  constexpr int kPiece = 32 * kDispatchU<V * sizeof(T)>;
  const int64_t gy = (a.cols / V + kPiece - 1) / kPiece;
  int64_t gx = (a.tokens + kWarps - 1) / kWarps;
  const int64_t padding = (padding_ctas(a.rows, kWarps) + gy - 1) / gy;
  if (gx < padding) gx = padding;
  if (gx > 0x7FFFFFFF || gy > 65535) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(gx), static_cast<unsigned>(gy));
  auto k = a.weights ? dispatch_kernel<T, V, true> : dispatch_kernel<T, V, false>;
  return launch(k, grid, kThreads, 1, 0, stream, rows_params(a));
}

template <typename T, int V, int kU, int kC>
cudaError_t launch_combine_u(const RowsArgs& a, cudaStream_t stream) {
  const int64_t gx = (a.tokens + kWarps - 1) / kWarps;
  const int64_t gy = (a.cols / V + 32 * kC - 1) / (32 * kC);
  if (gx > 0x7FFFFFFF || gy > 65535) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(gx), static_cast<unsigned>(gy));
  auto k = a.weights ? combine_kernel<T, V, true, kU, kC> : combine_kernel<T, V, false, kU, kC>;
  return launch(k, grid, kThreads, 1, 0, stream, rows_params(a));
}

// 8 accesses of a lane at once: of 8 rows, or of fewer and more columns where tokens have fewer.
template <typename T, int V>
cudaError_t launch_combine_v(const RowsArgs& a, cudaStream_t stream) {
  if constexpr (V * sizeof(T) == 16) {
    if (a.k <= 2) return launch_combine_u<T, V, 2, 4>(a, stream);
    if (a.k <= 4) return launch_combine_u<T, V, 4, 2>(a, stream);
    return launch_combine_u<T, V, 8, 1>(a, stream);
  } else {
    return launch_combine_u<T, V, 4, 8>(a, stream);
  }
}

template <typename T, int V, int kGroup, int kU, int kC>
cudaError_t launch_combine_grad_u(const RowsArgs& a, cudaStream_t stream) {
  constexpr int kPer = kGradThreads / kGroup;
  int64_t gx = (a.tokens + kPer - 1) / kPer;
  const int64_t padding = a.out ? padding_ctas(a.rows, kGradThreads / 32) : 0;
  if (gx < padding) gx = padding;
  if (gx > 0x7FFFFFFF) return cudaErrorInvalidValue;
  auto k = a.out ? combine_grad_kernel<T, V, kGroup, true, kU, kC>
                 : combine_grad_kernel<T, V, kGroup, false, kU, kC>;
  return launch(k, dim3(static_cast<unsigned>(gx)), kGradThreads, 1, 0, stream, rows_params(a));
}

// A warp a token where rows are short, else the CTA; a thread adds at most cols / 128 + 128
// products.
template <typename T, int V>
cudaError_t launch_combine_grad_v(const RowsArgs& a, cudaStream_t stream) {
  const bool narrow = a.cols / V <= 128;
  if constexpr (V * sizeof(T) == 16) {
    if (a.k <= 2)
      return a.cols / V <= 512 ? launch_combine_grad_u<T, V, 32, 2, 4>(a, stream)
                               : launch_combine_grad_u<T, V, kGradThreads, 2, 4>(a, stream);
    return narrow ? launch_combine_grad_u<T, V, 32, 8, 1>(a, stream)
                  : launch_combine_grad_u<T, V, kGradThreads, 8, 1>(a, stream);
  } else {
    return narrow ? launch_combine_grad_u<T, V, 32, 4, 4>(a, stream)
                  : launch_combine_grad_u<T, V, kGradThreads, 4, 4>(a, stream);
  }
}

// One launcher by the widest access that every row starts on (tensors start on 16 bytes).
#define MXFP8_BY_ACCESS(launcher, a, stream)                                              \
  do {                                                                                    \
    if ((a).fp32) {                                                                       \
      if ((a).cols % 4 == 0) return launcher<float, 4>(a, stream);                        \
      if ((a).cols % 2 == 0) return launcher<float, 2>(a, stream);                        \
      return launcher<float, 1>(a, stream);                                               \
    }                                                                                     \
    if ((a).cols % 8 == 0) return launcher<__nv_bfloat16, 8>(a, stream);                  \
    if ((a).cols % 4 == 0) return launcher<__nv_bfloat16, 4>(a, stream);                  \
    if ((a).cols % 2 == 0) return launcher<__nv_bfloat16, 2>(a, stream);                  \
    return launcher<__nv_bfloat16, 1>(a, stream);                                         \
  } while (0)

// Leave for the largest launch of route_kernel, asked for once a device. The attributes are the
// function's, not a launch's: one that followed each launch's own size would take leave away from
// another host thread's larger launch.
cudaError_t route_leave() {
  constexpr int kMost = static_cast<int>(
      sizeof(uint32_t) * kMaxExperts * kMaxRouteCtas +
      std::max(sizeof(uint32_t) * kMaxExperts * kRouteWarps,
               sizeof(uint2) * 32 * kBatch * kRouteWarps));
  static_assert(kMost + 9 * 1024 <= 227 * 1024, "with the static part, an SM's shared memory");
  static std::atomic<bool> given[64] = {};  // per device; asking twice is harmless
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool known = dev >= 0 && dev < 64;
  if (known && given[dev].load(std::memory_order_relaxed)) return cudaSuccess;
  e = cudaFuncSetAttribute(route_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(route_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  if (known) given[dev].store(true, std::memory_order_relaxed);
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_route(const RouteArgs& a, cudaStream_t stream) {
  RouteParams p{a.ids, a.entries, 0, a.num_experts, 0, a.rows, a.offsets, a.row_of, a.entry_of,
                a.status};
  while ((a.num_experts - 1) >> p.key_bits) ++p.key_bits;
  int ctas = 1;
  while (ctas < kMaxRouteCtas && a.entries > int64_t{1024} * ctas) ctas *= 2;
  const int64_t warps = static_cast<int64_t>(ctas) * kRouteWarps;
  p.per_warp = ((a.entries + warps - 1) / warps + 31) / 32 * 32;
  const size_t counters = sizeof(uint32_t) * a.num_experts * kRouteWarps;
  const size_t sorted = p.per_warp <= 32 * kBatch ? sizeof(uint2) * p.per_warp * kRouteWarps : 0;
  const size_t dyn = sizeof(uint32_t) * ((static_cast<size_t>(a.num_experts) * ctas + 3) / 4 * 4) +
                     std::max(counters, sorted);
  // Beyond 8 CTAs, the portable limit: 8192 x 8 entries of 128 experts take 8.5 us on 16 and 12.7
  // on 8, 16384 x 8 13.0 and 21.5, 1024 x 8 4.8 on 8. 48 KB without leave, the static part of 8.3 KB
  // among them.
  if (ctas > 8 || dyn > 32 * 1024) {
    const cudaError_t e = route_leave();
    if (e != cudaSuccess) return e;
  }
  return launch(route_kernel, dim3(static_cast<unsigned>(ctas)), kRouteThreads, ctas, dyn, stream,
                p);
}

cudaError_t launch_dispatch(const RowsArgs& a, cudaStream_t stream) {
  if (a.rows == 0 || a.cols == 0) return cudaSuccess;
  MXFP8_BY_ACCESS(launch_dispatch_v, a, stream);
}

cudaError_t launch_combine(const RowsArgs& a, cudaStream_t stream) {
  if (a.tokens == 0 || a.cols == 0) return cudaSuccess;
  MXFP8_BY_ACCESS(launch_combine_v, a, stream);
}

cudaError_t launch_combine_grad(const RowsArgs& a, cudaStream_t stream) {
  MXFP8_BY_ACCESS(launch_combine_grad_v, a, stream);
}

}  // namespace mxfp8
