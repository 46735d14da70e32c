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
constexpr int kMaxRouteCtas = 8;    // of the cluster (the portable limit)
constexpr int kBatch = 8;           // 32-entry groups whose ids a warp reads at once
static_assert(kMaxExperts <= kRouteThreads, "one thread an expert");

struct RouteParams {
  const int64_t* ids;
  int64_t n;            // entries
  int64_t per_warp;     // entries of a warp, a multiple of 32
  int E;
  int64_t rows;
  int32_t* offsets;
  int32_t* row_of;
  int32_t* entry_of;
  int* status;
};

// Stable counting sort by one cluster of CTAs. Each warp owns a contiguous run of entries: it
// counts them by expert in its own row of counters, a thread per expert turns the counters into
// places (over the warps of a CTA, then over the CTAs, whose totals go round through distributed
// shared memory), and each warp reads its entries again and hands out the places, 32 entries at
// a time in order. One launch, no workspace, and nothing depends on timing. Bound by latency: a
// chain of two reads of the ids, the counters and one cluster barrier.
__global__ void __launch_bounds__(kRouteThreads) route_kernel(const RouteParams p) {
  extern __shared__ uint32_t dyn[];
  uint32_t* count = dyn;                                  // [warps][E]
  uint32_t* total = dyn + kRouteWarps * p.E;              // [CTAs][E], every CTA's
  __shared__ uint32_t first_row[kMaxExperts];             // of this CTA's entries, by expert
  __shared__ uint32_t warp_sum[kRouteWarps];
  __shared__ uint32_t all_rows;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, E = p.E;
  const int ctas = static_cast<int>(gridDim.x), rank = static_cast<int>(blockIdx.x);
  for (int i = tid; i < kRouteWarps * E; i += kRouteThreads) count[i] = 0;
  if (ctas > 1) cluster_arrive();   // this CTA has started: its shared memory may be written
  __syncthreads();
  grid_dependency_wait();
  grid_launch_dependents();

  uint32_t* mine = count + warp * E;
  const int64_t begin = (static_cast<int64_t>(rank) * kRouteWarps + warp) * p.per_warp;
  const int64_t end = begin + p.per_warp < p.n ? begin + p.per_warp : p.n;
  int key[kBatch];   // the expert of the lane's entry in each group; -1 for none
  bool bad = false;
  const auto read = [&](int64_t at) {
#pragma unroll
    for (int g = 0; g < kBatch; ++g) {
      const int64_t i = at + 32 * g + lane;
      const int64_t id = i < end ? p.ids[i] : -1;
      bad |= id >= E;
      key[g] = id < 0 || id >= E ? -1 : static_cast<int>(id);
    }
  };
  for (int64_t at = begin; at < end; at += 32 * kBatch) {
    read(at);
#pragma unroll
    for (int g = 0; g < kBatch; ++g)
      if (key[g] >= 0) atomicAdd(mine + key[g], 1u);
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

  // segments: a scan over the experts of their counts, rounded up to 32
  uint32_t before = 0, all = 0;
  if (tid < E)
    for (int c = 0; c < ctas; ++c) {
      const uint32_t v = total[c * E + tid];
      before += c < rank ? v : 0;
      all += v;
    }
  const uint32_t padded = (all + 31u) & ~31u;
  uint32_t incl = padded;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t v = __shfl_up_sync(kFull, incl, d);
    if (lane >= d) incl += v;
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  uint32_t base = incl - padded;
  for (int w = 0; w < warp; ++w) base += warp_sum[w];
  if (tid == kRouteThreads - 1) all_rows = base + padded;
  __syncthreads();
  const bool fits = all_rows <= p.rows;   // n + 31 E is below 2^32: nothing wrapped
  if (tid < E) {
    first_row[tid] = base + before;
    // of the whole expert, for the padding below: end of its entries and of its segment
    total[tid] = base + all;
    if (rank == 0) p.offsets[tid] = fits ? static_cast<int32_t>(base) : 0;
  }
  if (rank == 0 && tid == 0) {
    p.offsets[E] = static_cast<int32_t>(p.rows);
    if (!fits) latch_error(p.status, MXFP8_ERR_BAD_OFFSETS);
  }
  __syncthreads();

  if (!fits) {   // a plan without entries: valid offsets, padding everywhere
    const int64_t step = static_cast<int64_t>(ctas) * kRouteThreads;
    for (int64_t i = static_cast<int64_t>(rank) * kRouteThreads + tid; i < p.n; i += step)
      p.row_of[i] = -1;
    for (int64_t r = static_cast<int64_t>(rank) * kRouteThreads + tid; r < p.rows; r += step)
      p.entry_of[r] = -1;
    return;
  }

  for (int64_t at = begin; at < end; at += 32 * kBatch) {
    if (p.per_warp > 32 * kBatch) read(at);   // else still there
#pragma unroll
    for (int g = 0; g < kBatch; ++g) {
      const int64_t i = at + 32 * g + lane;
      if (at + 32 * g >= end) break;          // the same in all lanes
      const unsigned same = __match_any_sync(kFull, key[g]);
      int32_t row = -1;
      if (key[g] >= 0)
        row = static_cast<int32_t>(first_row[key[g]] + mine[key[g]] +
                                   __popc(same & ((1u << lane) - 1u)));
      __syncwarp();
      if (key[g] >= 0 && (same >> lane) == 1u) mine[key[g]] += __popc(same);   // its last lane
      __syncwarp();
      if (i < end) p.row_of[i] = row;
      if (row >= 0) p.entry_of[row] = static_cast<int32_t>(i);
    }
  }
  // rows of no entry: the ends of the segments, and all that is left after the last
  for (int e = rank * kRouteWarps + warp; e < E; e += ctas * kRouteWarps) {
    const uint32_t r = total[e] + static_cast<uint32_t>(lane);
    if (r < ((total[e] + 31u) & ~31u)) p.entry_of[r] = -1;
  }
  for (int64_t r = static_cast<int64_t>(all_rows) + rank * kRouteThreads + tid; r < p.rows;
       r += static_cast<int64_t>(ctas) * kRouteThreads)
    p.entry_of[r] = -1;
}

// ------------------------------------------------------------------ values of a row

// V consecutive elements of a row, moved as one access of kBytes and computed with in FP32.
template <int kBytes>
struct Raw;
template <>
struct Raw<16> { using type = uint4; };
template <>
struct Raw<4> { using type = uint32_t; };
template <>
struct Raw<2> { using type = uint16_t; };

template <typename T, int V>
struct Pack {
  using raw = typename Raw<V * static_cast<int>(sizeof(T))>::type;
};

__device__ __forceinline__ uint4 load_once(const uint4* p) { return ld_nc_v4(p); }
__device__ __forceinline__ uint32_t load_once(const uint32_t* p) { return __ldg(p); }
__device__ __forceinline__ uint16_t load_once(const uint16_t* p) { return __ldg(p); }

__device__ __forceinline__ void zero(uint4& v) { v = make_uint4(0, 0, 0, 0); }
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
      w[i] = sizeof(T) == 4 ? __float_as_uint(x[i]) : cvt_bf16x2(x[(2 * i + 1) % V], x[(2 * i) % V]);
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

// Rows without an entry in every 32-row group that falls to this CTA, set to zero by its warps.
template <typename T, int V>
__device__ __forceinline__ void zero_padding(const RowsParams& p, int64_t cta, int64_t ctas,
                                             int warps) {
  using raw = typename Pack<T, V>::raw;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  raw none;
  zero(none);
  const int64_t vecs = p.cols / V;
  for (int64_t r0 = 32 * cta; r0 < p.rows; r0 += 32 * ctas) {   // rows: a multiple of 32
    unsigned pad = __ballot_sync(kFull, p.entry_of[r0 + lane] < 0);
    for (int at = 0; pad; pad &= pad - 1, ++at) {
      if (at % warps != warp) continue;
      raw* out = reinterpret_cast<raw*>(p.out) + (r0 + __ffs(pad) - 1) * vecs;
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

// A warp reads a piece of a token's row once and writes it to the token's k rows; the rows of
// no entry are zeroed on the side. Bound by the writes.
template <typename T, int V, bool kWeighted>
__global__ void __launch_bounds__(kThreads) dispatch_kernel(const RowsParams p) {
  using raw = typename Pack<T, V>::raw;
  constexpr int kU = 4;
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  const int64_t vecs = p.cols / V;
  const int64_t c0 = static_cast<int64_t>(blockIdx.y) * 32 * kU + lane;
  if (t < p.tokens) {
    const raw* x = reinterpret_cast<const raw*>(p.src) + t * vecs;
    raw v[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u)
      if (c0 + 32 * u < vecs) v[u] = load_once(x + c0 + 32 * u);
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
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          if (c0 + 32 * u >= vecs) continue;
          if constexpr (kWeighted) {
            float f[V];
            unpack<T, V>(v[u], f);
#pragma unroll
            for (int i = 0; i < V; ++i) f[i] = __fmul_rn(f[i], w);
            out[c0 + 32 * u] = pack<T, V>(f);
          } else {
            out[c0 + 32 * u] = v[u];
          }
        }
      }
    }
  }
  const int64_t ctas = static_cast<int64_t>(gridDim.x) * gridDim.y;
  zero_padding<T, V>(p, static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x, ctas, kWarps);
}

// ------------------------------------------------------------------------------- combine

// A warp sums a piece (32 lanes x V columns) of a token's k rows. Bound by the reads.
template <typename T, int V, bool kWeighted>
__global__ void __launch_bounds__(kThreads) combine_kernel(const RowsParams p) {
  using raw = typename Pack<T, V>::raw;
  constexpr int kU = 8;   // rows read at once
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  const int64_t vecs = p.cols / V;
  const int64_t c = static_cast<int64_t>(blockIdx.y) * 32 + lane;
  if (t >= p.tokens) return;
  const raw* y = reinterpret_cast<const raw*>(p.src);
  float sum[V];
#pragma unroll
  for (int i = 0; i < V; ++i) sum[i] = 0.f;
  for (int j0 = 0; j0 < p.k; j0 += 32) {
    const int left = p.k - j0 < 32 ? p.k - j0 : 32;
    int32_t my_row = -1;
    float my_w = 1.f;
    if (lane < left) {
      my_row = plan_row(p, t * p.k + j0 + lane);
      if (kWeighted && my_row >= 0) my_w = p.weights[t * p.k + j0 + lane];
    }
    for (int j = 0; j < left; j += kU) {
      raw v[kU];
      int32_t r[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        r[u] = __shfl_sync(kFull, my_row, (j + u) & 31);
        if (j + u >= left) r[u] = -1;
        if (r[u] >= 0 && c < vecs) v[u] = load_once(y + r[u] * vecs + c);
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const float w = kWeighted ? __shfl_sync(kFull, my_w, (j + u) & 31) : 1.f;
        if (r[u] < 0 || c >= vecs) continue;
        float f[V];
        unpack<T, V>(v[u], f);
#pragma unroll
        for (int i = 0; i < V; ++i) sum[i] = kWeighted ? fmaf(w, f[i], sum[i]) : sum[i] + f[i];
      }
    }
  }
  if (c < vecs) reinterpret_cast<raw*>(p.out)[t * vecs + c] = pack<T, V>(sum);
}

// -------------------------------------------------------------------- combine's gradient

constexpr int kGradThreads = 128;
constexpr int kGradU = 8;   // rows of a token at once

// A group of kGroup threads (a warp, or the CTA) takes a token: it reads dout[t] and the token's
// rows of y, writes w dout[t] to the rows' gradients and sums the products for the weights'. The
// sums are joined over the lanes, then over the warps in order. Bound by memory.
template <typename T, int V, int kGroup, bool kRows>
__global__ void __launch_bounds__(kGradThreads) combine_grad_kernel(const RowsParams p) {
  using raw = typename Pack<T, V>::raw;
  __shared__ float part[kGradThreads / 32][kGradU];
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
  for (int j0 = 0; j0 < p.k; j0 += kGradU) {
    int32_t r[kGradU];
    float w[kGradU], dot[kGradU];
#pragma unroll
    for (int u = 0; u < kGradU; ++u) {
      const bool there = live && j0 + u < p.k;
      r[u] = there ? plan_row(p, t * p.k + j0 + u) : -1;
      w[u] = r[u] >= 0 ? p.weights[t * p.k + j0 + u] : 0.f;
      dot[u] = 0.f;
    }
    if (live) {
      for (int64_t c = in_group; c < vecs; c += kGroup) {
        float gv[V];
        raw v[kGradU];
        unpack<T, V>(load_once(g + c), gv);
#pragma unroll
        for (int u = 0; u < kGradU; ++u)
          if (r[u] >= 0) v[u] = load_once(y + r[u] * vecs + c);
#pragma unroll
        for (int u = 0; u < kGradU; ++u) {
          if (r[u] < 0) continue;
          float f[V];
          unpack<T, V>(v[u], f);
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
#pragma unroll
    for (int u = 0; u < kGradU; ++u)
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) dot[u] += __shfl_xor_sync(kFull, dot[u], d);
    if constexpr (kGroup == 32) {
      if (live && lane == 0)
#pragma unroll
        for (int u = 0; u < kGradU; ++u)
          if (j0 + u < p.k) p.grad_w[t * p.k + j0 + u] = dot[u];
    } else {
      if (lane == 0)
#pragma unroll
        for (int u = 0; u < kGradU; ++u) part[warp][u] = dot[u];
      __syncthreads();
      if (threadIdx.x < kGradU && j0 + static_cast<int>(threadIdx.x) < p.k) {
        float sum = 0.f;
#pragma unroll
        for (int q = 0; q < kGradThreads / 32; ++q) sum += part[q][threadIdx.x];
        p.grad_w[t * p.k + j0 + threadIdx.x] = sum;
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

// Elements of an access: 16 bytes where every row starts on 16 bytes (tensors do), else one.
template <typename T>
bool whole_vectors(int64_t cols) {
  return cols * static_cast<int64_t>(sizeof(T)) % 16 == 0;
}

template <typename T, int V>
cudaError_t launch_dispatch_v(const RowsArgs& a, cudaStream_t stream) {
  const int64_t gx = (a.tokens + kWarps - 1) / kWarps;
  const int64_t gy = (a.cols / V + 127) / 128;
  if (gx > 0x7FFFFFFF || gy > 65535) return cudaErrorInvalidValue;
  // at least one CTA: a plan of no tokens is all padding
  const dim3 grid(static_cast<unsigned>(gx ? gx : 1), static_cast<unsigned>(gy));
  auto k = a.weights ? dispatch_kernel<T, V, true> : dispatch_kernel<T, V, false>;
  return launch(k, grid, kThreads, 1, 0, stream, rows_params(a));
}

template <typename T, int V>
cudaError_t launch_combine_v(const RowsArgs& a, cudaStream_t stream) {
  const int64_t gx = (a.tokens + kWarps - 1) / kWarps;
  const int64_t gy = (a.cols / V + 31) / 32;
  if (gx > 0x7FFFFFFF || gy > 65535) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(gx), static_cast<unsigned>(gy));
  auto k = a.weights ? combine_kernel<T, V, true> : combine_kernel<T, V, false>;
  return launch(k, grid, kThreads, 1, 0, stream, rows_params(a));
}

template <typename T, int V>
cudaError_t launch_combine_grad_v(const RowsArgs& a, cudaStream_t stream) {
  const bool narrow = a.cols / V <= 128;   // a warp a token
  const int per = narrow ? kGradThreads / 32 : 1;
  int64_t gx = (a.tokens + per - 1) / per;
  if (gx > 0x7FFFFFFF) return cudaErrorInvalidValue;
  if (gx == 0) gx = 1;
  auto k = narrow ? (a.out ? combine_grad_kernel<T, V, 32, true>
                           : combine_grad_kernel<T, V, 32, false>)
                  : (a.out ? combine_grad_kernel<T, V, kGradThreads, true>
                           : combine_grad_kernel<T, V, kGradThreads, false>);
  return launch(k, dim3(static_cast<unsigned>(gx)), kGradThreads, 1, 0, stream, rows_params(a));
}

}  // namespace

cudaError_t launch_route(const RouteArgs& a, cudaStream_t stream) {
  RouteParams p{a.ids, a.entries, 0, a.num_experts, a.rows, a.offsets, a.row_of, a.entry_of,
                a.status};
  int ctas = 1;
  while (ctas < kMaxRouteCtas && a.entries > int64_t{4096} * ctas) ctas *= 2;
  const int64_t warps = static_cast<int64_t>(ctas) * kRouteWarps;
  p.per_warp = ((a.entries + warps - 1) / warps + 31) / 32 * 32;
  const size_t dyn = sizeof(uint32_t) * static_cast<size_t>(a.num_experts) * (kRouteWarps + ctas);
  if (dyn > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(
        route_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(dyn));
    if (e != cudaSuccess) return e;
  }
  return launch(route_kernel, dim3(static_cast<unsigned>(ctas)), kRouteThreads, ctas, dyn, stream,
                p);
}

cudaError_t launch_dispatch(const RowsArgs& a, cudaStream_t stream) {
  if (a.rows == 0 || a.cols == 0) return cudaSuccess;
  if (a.fp32)
    return whole_vectors<float>(a.cols) ? launch_dispatch_v<float, 4>(a, stream)
                                        : launch_dispatch_v<float, 1>(a, stream);
  return whole_vectors<__nv_bfloat16>(a.cols) ? launch_dispatch_v<__nv_bfloat16, 8>(a, stream)
                                              : launch_dispatch_v<__nv_bfloat16, 1>(a, stream);
}

cudaError_t launch_combine(const RowsArgs& a, cudaStream_t stream) {
  if (a.tokens == 0 || a.cols == 0) return cudaSuccess;
  if (a.fp32)
    return whole_vectors<float>(a.cols) ? launch_combine_v<float, 4>(a, stream)
                                        : launch_combine_v<float, 1>(a, stream);
  return whole_vectors<__nv_bfloat16>(a.cols) ? launch_combine_v<__nv_bfloat16, 8>(a, stream)
                                              : launch_combine_v<__nv_bfloat16, 1>(a, stream);
}

cudaError_t launch_combine_grad(const RowsArgs& a, cudaStream_t stream) {
  if (a.fp32)
    return whole_vectors<float>(a.cols) ? launch_combine_grad_v<float, 4>(a, stream)
                                        : launch_combine_grad_v<float, 1>(a, stream);
  return whole_vectors<__nv_bfloat16>(a.cols) ? launch_combine_grad_v<__nv_bfloat16, 8>(a, stream)
                                              : launch_combine_grad_v<__nv_bfloat16, 1>(a, stream);
}

}  // namespace mxfp8
