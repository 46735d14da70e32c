// logprob.cu - log probabilities of given tokens, with the entropy and the likeliest
// alternatives of each row of logits, and the gradient of all three.
//
// The quantity by which "End-to-End MXFP8 RL on Blackwell" (verl blog post) compares a
// sampler with a learner (section "A different grid, and drift") and on which the learner's
// policy gradient acts: the log probability that a row of logits gives to a token.
//
// With m = max x, d = (x - m) / T and S = sum e^d:
//   log p_v = d_v - log S,   H = -sum p log p = log S - sum(e^d d) / S.
// Everything is taken relative to the row's maximum, so no large log-sum-exp is subtracted
// from a large logit. Sums, maxima and statistics are FP32. A thread adds up at most max(256,
// vocab / 256) values in order (an eighth of that where 8 CTAs share a row), then threads and
// CTAs are joined pairwise, so log S is off by at most (that number + 64) 2^-24 + 2^-20. Powers are
// taken in base 2: one multiplication by log2(e) / T, then ex2.approx, which is 2^-22 off at most
// and takes one instruction: a choice for speed, well inside that bound.
//
// Masks: a logit of -inf (or one so far below the maximum that e^d vanishes, such as the
// type's lowest value) has probability 0 and adds nothing to the entropy. t = d log2(e) is
// clamped at -256, where 2^t is already 0 in FP32, so that 0 * -inf never arises. A row
// whose logits are all -inf has no distribution: log probability -inf, entropy 0, no
// alternatives, zero gradient. A row that holds a NaN or +inf gives NaN.

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "device.cuh"
#include "internal.h"
#include "mxfp8.h"

namespace mxfp8 {
namespace {

constexpr int kThreads = 256;  // of the gradient kernel, and the most of the forward one
constexpr int kMaxSplit = 8;   // CTAs of a cluster that share one row (the portable limit)
constexpr int kMaxTop = 32;    // alternatives: one per lane of a warp's list
constexpr float kLowest = -256.f;  // 2^t is 0 from here on
constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.693147180559945309f;
constexpr float kInf = __builtin_huge_valf();

__device__ __forceinline__ float max_nan(float a, float b) {  // NaN wins
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

__device__ __forceinline__ float ex2(float t) {
  float d;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(d) : "f"(t));
  return d;
}

// 16 bytes of logits as FP32 values.
template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int kN = 4;
  static __device__ __forceinline__ void unpack(const uint4& w, float (&x)[4]) {
    x[0] = __uint_as_float(w.x);
    x[1] = __uint_as_float(w.y);
    x[2] = __uint_as_float(w.z);
    x[3] = __uint_as_float(w.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&x)[4]) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                      __float_as_uint(x[3]));
  }
  static __device__ __forceinline__ float load(const float* p) { return *p; }
  static __device__ __forceinline__ void store(float* p, float v) { *p = v; }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int kN = 8;
  static __device__ __forceinline__ void unpack(const uint4& w, float (&x)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(u[i] << 16);
      x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&x)[8]) {
    return make_uint4(cvt_bf16x2(x[1], x[0]), cvt_bf16x2(x[3], x[2]), cvt_bf16x2(x[5], x[4]),
                      cvt_bf16x2(x[7], x[6]));
  }
  static __device__ __forceinline__ float load(const __nv_bfloat16* p) {
    return __bfloat162float(*p);
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, float v) {
    *p = __float2bfloat16_rn(v);
  }
};

// Where the 16-byte vectors of a row lie: `head` single values up to the first 16-byte
// boundary, `nv` vectors, then `tail` single values. A row of an odd vocabulary starts on
// any element.
struct RowShape {
  int head, tail;
  int64_t nv;
};

template <typename T>
__device__ __forceinline__ RowShape row_shape(const T* row, int64_t vocab) {
  constexpr int kN = Vec<T>::kN;
  const int off = static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T));
  RowShape s;
  int64_t h = off ? kN - off : 0;
  h = h < vocab ? h : vocab;
  s.head = static_cast<int>(h);
  s.nv = (vocab - h) / kN;
  s.tail = static_cast<int>(vocab - h - s.nv * kN);
  return s;
}

// The running maximum, sum and weighted sum of a softmax: m, S = sum 2^t, E = sum 2^t t,
// with t = (x - m) c; `sub` is m, or 0 while nothing above -inf has been seen.
struct Softmax {
  float m = -kInf, sub = 0.f, s = 0.f, e = 0.f;

  // what has been summed so far, relative to a new maximum
  __device__ __forceinline__ void raise(float to, float c) {
    const float delta = m == -kInf ? kLowest : max_nan((sub - to) * c, kLowest);
    const float a = ex2(delta);
    e = a * fmaf(delta, s, e);
    s *= a;
    m = sub = to;
  }

  // adds kN values; returns their maximum
  template <int kN>
  __device__ __forceinline__ float add(const float (&x)[kN], float c) {
    float top = x[0];
#pragma unroll
    for (int i = 1; i < kN; ++i) top = fmaxf(top, x[i]);
    if (top > m) raise(top, c);
    const uint64_t neg = pack2(-sub, -sub), cc = pack2(c, c);
    uint64_t s2 = pack2(s, 0.f), e2 = pack2(e, 0.f);
#pragma unroll
    for (int i = 0; i < kN; i += 2) {
      float t0, t1;
      unpack2(mul2(add2(pack2(x[i], x[i + 1]), neg), cc), t0, t1);
      t0 = max_nan(t0, kLowest);
      t1 = max_nan(t1, kLowest);
      const uint64_t p = pack2(ex2(t0), ex2(t1));
      s2 = add2(s2, p);
      e2 = fma2(p, pack2(t0, t1), e2);
    }
    float a, b;
    unpack2(s2, a, b);
    s = a + b;
    unpack2(e2, a, b);
    e = a + b;
    return top;
  }

  __device__ __forceinline__ void join(float om, float os, float oe, float c) {
    const float top = fmaxf(m, om);
    if (top > m) raise(top, c);
    const float delta = om == -kInf ? kLowest : max_nan((om - sub) * c, kLowest);
    const float a = ex2(delta);
    e += a * fmaf(delta, os, oe);
    s += a * os;
  }
};

// ------------------------------------------------------------------- alternatives (top k)
// An alternative is a 64-bit key: the value's bits in an order-preserving form, then the
// complement of its place, so that the largest key is the largest value at the lowest
// place. -0 counts as 0. Keys at or below kNoKey (-inf and lower) are not alternatives.
constexpr uint64_t kNoKey = 0x007FFFFFFFFFFFFFull;

__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint64_t key) {
  const uint32_t o = static_cast<uint32_t>(key >> 32);
  return __uint_as_float((o & 0x80000000u) ? o & 0x7FFFFFFFu : ~o);
}
__device__ __forceinline__ uint64_t key_of(float x, uint32_t place) {
  return (static_cast<uint64_t>(order_of(x)) << 32) | (0xFFFFFFFFu - place);
}

// A warp's k best keys, lane l holding the l-th. `least` is what a key has to beat.
struct WarpTop {
  uint64_t mine = kNoKey, least;

  // every lane offers one key (kNoKey for none)
  __device__ __forceinline__ void offer(uint64_t key, int k, int lane) {
    uint32_t want = __ballot_sync(0xFFFFFFFFu, key > least);
    while (want) {
      const int src = __ffs(want) - 1;
      const uint64_t cand = __shfl_sync(0xFFFFFFFFu, key, src);
      const int at = __popc(__ballot_sync(0xFFFFFFFFu, mine > cand));
      const uint64_t up = __shfl_up_sync(0xFFFFFFFFu, mine, 1);
      if (lane >= at) mine = lane == at ? cand : up;
      const uint64_t last = __shfl_sync(0xFFFFFFFFu, mine, k - 1);
      least = last > least ? last : least;
      if (lane == src) key = kNoKey;
      want = __ballot_sync(0xFFFFFFFFu, key > least);
    }
  }
};

constexpr int kMaxCandidates = 512;

template <int kThreads>
struct Shared {
  static constexpr int kWarps = kThreads / 32;
  float part[kWarps][3];            // the warps' m, S, E
  float parts[kMaxSplit][3];        // first CTA of a cluster: the CTAs' m, S, E
  float row[2];                     // the row's maximum and log S
  uint32_t warp_bar[kWarps];        // order of each warp's j-th largest thread maximum
  int chosen[kThreads];             // threads whose largest value reaches the bar
  int reread[kThreads];             // and of those, the ones whose second vector does too
  int num_chosen, num_reread, num_candidates;
  uint64_t keys[kMaxCandidates];    // candidates; then lists to be merged
  uint64_t lists[kMaxSplit * kMaxTop];  // first CTA of a cluster: the CTAs' best keys
  uint64_t top[kMaxTop];            // the best keys, in order
};

// The k largest of keys [0, n), in order, into `out`, which the caller has filled with kNoKey
// (it stays where fewer exist). Keys are distinct but for kNoKey. Called by the whole CTA;
// `out` is ready after the next barrier.
template <int kThreads>
__device__ __forceinline__ void rank_keys(const uint64_t* keys, int n, int k, uint64_t* out,
                                          int tid) {
  for (int t = tid; t < n; t += kThreads) {
    const uint64_t mine = keys[t];
    int above = 0;
#pragma unroll 4
    for (int i = 0; i < n; ++i) above += keys[i] > mine;
    if (mine > kNoKey && above < k) out[above] = mine;
  }
}

struct Params {
  const void* logits;
  int64_t rows, vocab, ld;
  const int64_t* targets;
  float inv_t;
  float* logprob;
  float* entropy;
  float* stats;
  int top;
  float* top_logprob;
  int64_t* top_id;
  int* status;
};

// What the stream keeps for the alternatives, of a thread's vectors: the largest value and
// which vector holds it, and the largest value of the other vectors.
struct Best {
  float top = -kInf, second = -kInf;
  uint32_t at = 0;  // relative to the CTA's first vector

  __device__ __forceinline__ void add(float x, uint32_t v) {
    second = fmaxf(second, fminf(x, top));
    at = x > top ? v : at;
    top = fmaxf(top, x);
  }
};

// The CTA's k best keys into sh.top, from what its threads kept of their vectors (v0 + tid + i
// kThreads) and from its single values.
//
// A bar that at least k of the threads' largest values reach bounds the k-th best value from
// below, so the values that reach it are all there is to look at. The bar is the smallest,
// over the warps with values in every lane, of the warp's j-th largest maximum, with j such
// that those are k values in all: for k = 8 about 20 values of a row reach it. Most are alone
// in their thread, which reads the vector that holds it once more. Only a thread whose second
// vector reaches the bar too has all its vectors read again. (Reading all vectors of every
// thread that reaches the bar took 46% longer at 4096 x 131072: 32-byte pieces 4 KB apart.)
// What reaches the bar is listed, and ranked by counting; where it is more than the list holds
// (many equal values), sorted lists kept by the warps take over.
// A barrier stands between the two halves.
template <int kThreads>
__device__ __forceinline__ void set_bars(Shared<kThreads>& sh, int64_t v0, int64_t v1,
                                         const Best& kept, int k) {
  constexpr int kWarps = kThreads / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t full = (v1 - v0) / 32;  // warps with a vector in every lane
  const int warps = static_cast<int>(full < kWarps ? full : kWarps);
  if (warps > 0 && 32 * warps >= k) {
    const int j = (k + warps - 1) / warps;
    uint32_t v = order_of(kept.top), best = 0;
    for (int i = 0; i < j; ++i) {
      best = __reduce_max_sync(0xFFFFFFFFu, v);
      const int at = __ffs(__ballot_sync(0xFFFFFFFFu, v == best)) - 1;
      if (lane == at) v = 0;
    }
    if (lane == 0) sh.warp_bar[warp] = best;
  }
  if (tid == 0) sh.num_chosen = sh.num_reread = sh.num_candidates = 0;
  if (tid < k) sh.top[tid] = kNoKey;
}

template <int kThreads, typename T>
__device__ __forceinline__ void find_top(Shared<kThreads>& sh, const T* row, const RowShape& shape,
                                         int64_t v0, int64_t v1, bool first, bool last,
                                         const Best& kept, int k) {
  constexpr int kN = Vec<T>::kN, kWarps = kThreads / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint4* body = reinterpret_cast<const uint4*>(row + shape.head);
  const int64_t tail0 = shape.head + shape.nv * kN;
  constexpr uint32_t kNone = static_cast<uint32_t>(kNoKey >> 32);  // order of -inf
  const uint32_t own = order_of(kept.top);
  const int64_t full = (v1 - v0) / 32;
  const int warps = static_cast<int>(full < kWarps ? full : kWarps);
  uint32_t bar_order = kNone + 1;
  if (warps > 0 && 32 * warps >= k) {
    uint32_t least = 0xFFFFFFFFu;
    for (int w = 0; w < warps; ++w) least = min(least, sh.warp_bar[w]);
    bar_order = max(least, kNone + 1);
  }
  const float bar = value_of(static_cast<uint64_t>(bar_order) << 32);
  auto list = [&](float x, int64_t place) {
    if (!(x >= bar)) return;
    const int at = atomicAdd(&sh.num_candidates, 1);
    if (at < kMaxCandidates) sh.keys[at] = key_of(x, static_cast<uint32_t>(place));
  };
  auto list_vector = [&](const uint4& w, int64_t v) {
    float x[kN];
    Vec<T>::unpack(w, x);
#pragma unroll
    for (int i = 0; i < kN; ++i) list(x[i], shape.head + v * kN + i);
  };
  if (own >= bar_order) {
    sh.chosen[atomicAdd(&sh.num_chosen, 1)] = tid;
    if (order_of(kept.second) >= bar_order) sh.reread[atomicAdd(&sh.num_reread, 1)] = tid;
    else list_vector(__ldg(body + v0 + kept.at), v0 + kept.at);
  }
  const bool has_head = first && tid < shape.head, has_tail = last && tid < shape.tail;
  if (has_head) list(Vec<T>::load(row + tid), tid);
  if (has_tail) list(Vec<T>::load(row + tail0 + tid), tail0 + tid);
  __syncthreads();
  const int steps = static_cast<int>((v1 - v0 + kThreads - 1) / kThreads);
  const int runs = (steps + 31) / 32;  // of 32 vectors, one a lane, for each thread
  const int all = sh.num_reread * runs;  // the same for every thread
  for (int g = warp; g < all; g += kWarps) {
    const int c = g / runs;
    const int64_t v = v0 + sh.reread[c] + static_cast<int64_t>((g - c * runs) * 32 + lane) * kThreads;
    if (v < v1) list_vector(__ldg(body + v), v);
  }
  if (all > 0) __syncthreads();
  int listed = sh.num_candidates;
  if (listed > kMaxCandidates) {
    __syncthreads();
    const int n = sh.num_chosen;
    WarpTop best;
    best.least = bar_order > kNone + 1 ? (static_cast<uint64_t>(bar_order) << 32) - 1 : kNoKey;
    for (int q = warp; q < n; q += kWarps) {
      const int owner = sh.chosen[q];
      for (int r = 0; r < runs; ++r) {
        const int64_t v = v0 + owner + static_cast<int64_t>(r * 32 + lane) * kThreads;
        const bool live = v < v1;
        float x[kN];
        Vec<T>::unpack(live ? __ldg(body + v) : make_uint4(0, 0, 0, 0), x);
#pragma unroll 1
        for (int i = 0; i < kN; ++i) {
          float xi = x[0];
#pragma unroll
          for (int e = 1; e < kN; ++e) xi = e == i ? x[e] : xi;
          best.offer(live ? key_of(xi, static_cast<uint32_t>(shape.head + v * kN + i)) : kNoKey,
                     k, lane);
        }
      }
    }
    if (warp == 0) {  // the single values, fewer than 8 on either side
      uint64_t key = kNoKey;
      if (has_head) key = key_of(Vec<T>::load(row + lane), static_cast<uint32_t>(lane));
      best.offer(key, k, lane);
      key = kNoKey;
      if (has_tail) key = key_of(Vec<T>::load(row + tail0 + lane), static_cast<uint32_t>(tail0 + lane));
      best.offer(key, k, lane);
    }
    sh.keys[warp * kMaxTop + lane] = lane < k ? best.mine : kNoKey;
    listed = kWarps * kMaxTop;
    __syncthreads();
  }
  rank_keys<kThreads>(sh.keys, listed, k, sh.top, tid);
  __syncthreads();
}

// One cluster of `split` CTAs per row; each CTA streams a contiguous part of it once.
//
// Bound by memory (2 or 4 bytes a logit): 16-byte loads, four of them in flight a thread, each
// logit read once. 4096 x 131072 BF16: 159 us (6.7 TB/s), 179 with the 8 likeliest tokens. One
// row of 131072 takes 4.1 us, 7.2 with the 5 likeliest, 8.7 with 20.
// Rows are split over a cluster only when there are too few of them to fill the GPU; each
// CTA then hands its sums and best keys to the first through distributed shared memory,
// without a workspace.
template <typename T, bool kTop, int kThreads>
__global__ void __launch_bounds__(kThreads)
logprob_kernel(const Params p, int split) {
  constexpr int kN = Vec<T>::kN, kWarps = kThreads / 32;
  constexpr int kUnroll = 4;
  __shared__ Shared<kThreads> sh;
  if (split > 1) cluster_arrive();  // this CTA has started: its shared memory may be written
  grid_dependency_wait();
  grid_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row_id = blockIdx.x / static_cast<unsigned>(split);
  const int rank = static_cast<int>(blockIdx.x % static_cast<unsigned>(split));
  const T* row = static_cast<const T*>(p.logits) + row_id * p.ld;
  const RowShape shape = row_shape(row, p.vocab);
  const int64_t v0 = shape.nv * rank / split, v1 = shape.nv * (rank + 1) / split;
  const uint4* body = reinterpret_cast<const uint4*>(row + shape.head);
  const bool first = rank == 0, last = rank == split - 1;
  const bool has_head = first && tid < shape.head, has_tail = last && tid < shape.tail;
  const int64_t tail0 = shape.head + shape.nv * kN;
  const float c = p.inv_t * kLog2e;
  // thread 0 of the first CTA will need the target's logit
  int64_t target = 0;
  float target_logit = 0.f;
  if (first && tid == 0) {
    target = p.targets[row_id];
    if (target >= 0 && target < p.vocab) target_logit = Vec<T>::load(row + target);
  }

  Softmax sm;
  Best kept;
  int64_t v = v0 + tid;
  for (; v + (kUnroll - 1) * kThreads < v1; v += kUnroll * kThreads) {
    uint4 w[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) w[u] = ld_nc_v4(body + v + u * kThreads);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      float x[kN];
      Vec<T>::unpack(w[u], x);
      const float top = sm.add(x, c);
      if constexpr (kTop) kept.add(top, static_cast<uint32_t>(v - v0) + u * kThreads);
    }
  }
  for (; v < v1; v += kThreads) {
    float x[kN];
    Vec<T>::unpack(ld_nc_v4(body + v), x);
    const float top = sm.add(x, c);
    if constexpr (kTop) kept.add(top, static_cast<uint32_t>(v - v0));
  }
  if (has_head || has_tail) {
    const float x[2] = {has_head ? Vec<T>::load(row + tid) : -kInf,
                        has_tail ? Vec<T>::load(row + tail0 + tid) : -kInf};
    sm.add(x, c);
  }
  // join the CTA's threads
  auto join_lanes = [&](int lanes) {
    for (int o = lanes / 2; o > 0; o >>= 1) {
      const float om = __shfl_xor_sync(0xFFFFFFFFu, sm.m, o);
      const float os = __shfl_xor_sync(0xFFFFFFFFu, sm.s, o);
      const float oe = __shfl_xor_sync(0xFFFFFFFFu, sm.e, o);
      sm.join(om, os, oe, c);
    }
  };
  join_lanes(32);
  if constexpr (kTop) set_bars(sh, v0, v1, kept, p.top);
  if (lane == 0) {
    sh.part[warp][0] = sm.m;
    sh.part[warp][1] = sm.s;
    sh.part[warp][2] = sm.e;
  }
  __syncthreads();
  if (warp == 0) {
    sm.m = sh.part[lane % kWarps][0];
    sm.s = sh.part[lane % kWarps][1];
    sm.e = sh.part[lane % kWarps][2];
    sm.sub = sm.m == -kInf ? 0.f : sm.m;
    join_lanes(kWarps);
  }
  if constexpr (kTop) find_top(sh, row, shape, v0, v1, first, last, kept, p.top);

  // join the cluster's CTAs in its first
  if (split > 1) {
    cluster_wait();
    const uint32_t dst = 0;
    if (tid == 0) {
      const float o[3] = {sm.m, sm.s, sm.e};
      for (int i = 0; i < 3; ++i)
        st_cluster_u32(cluster_map(&sh.parts[rank][i], dst), __float_as_uint(o[i]));
    }
    if constexpr (kTop) {
      if (tid < p.top) {
        const uint64_t key = sh.top[tid];
        const uint32_t to = cluster_map(&sh.lists[rank * p.top + tid], dst);
        asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(to), "l"(key) : "memory");
      }
    }
    cluster_arrive();
    cluster_wait();
    if (rank != 0) return;
    if (warp == 0) {
      const int r = lane % kMaxSplit;
      sm.m = r < split ? sh.parts[r][0] : -kInf;
      sm.s = r < split ? sh.parts[r][1] : 0.f;
      sm.e = r < split ? sh.parts[r][2] : 0.f;
      sm.sub = sm.m == -kInf ? 0.f : sm.m;
      join_lanes(kMaxSplit);
    }
    if constexpr (kTop) {
      if (tid < p.top) sh.top[tid] = kNoKey;  // its own keys have been read into the lists
      __syncthreads();
      rank_keys<kThreads>(sh.lists, split * p.top, p.top, sh.top, tid);
      __syncthreads();
    }
  }

  if (tid == 0) {
    const float m = sm.m, s = sm.s, e = sm.e;
    const bool empty = m == -kInf && s == 0.f;  // every logit -inf (a NaN makes s NaN)
    const float log_s = empty ? 0.f : logf(s);
    float lp = 0.f;
    if (target >= p.vocab) {
      latch_error(p.status, MXFP8_ERR_BAD_TARGET);
      lp = __uint_as_float(0x7FC00000u);
    } else if (target >= 0) {
      lp = empty ? -kInf : (target_logit - m) * p.inv_t - log_s;
    }
    if (isnan(s)) lp = s;
    const float row_max = isnan(s) ? s : m;
    p.logprob[row_id] = lp;
    p.entropy[row_id] = empty ? 0.f : log_s - kLn2 * e / s;
    p.stats[2 * row_id] = row_max;
    p.stats[2 * row_id + 1] = log_s;
    sh.row[0] = row_max;
    sh.row[1] = log_s;
  }
  if constexpr (kTop) {
    __syncthreads();
    if (tid < p.top) {
      const uint64_t key = sh.top[tid];
      const bool none = key <= kNoKey || isnan(sh.row[1]);
      const float lp = (value_of(key) - sh.row[0]) * p.inv_t - sh.row[1];
      p.top_logprob[row_id * p.top + tid] = isnan(sh.row[1]) ? sh.row[1] : none ? -kInf : lp;
      p.top_id[row_id * p.top + tid] =
          none ? -1 : static_cast<int64_t>(0xFFFFFFFFu - static_cast<uint32_t>(key));
    }
  }
}

struct GradParams {
  const void* logits;
  int64_t rows, vocab, ld;
  const int64_t* targets;
  float inv_t;
  const float* stats;
  const float* entropy;
  const float* g_logprob;
  const float* g_entropy;  // or null
  int top;
  const int64_t* top_id;
  const float* g_top;
  void* out;
  int64_t out_ld;
  int64_t per_cta;         // vectors (or single values) of a row that one CTA handles
  int parts;               // CTAs per row
  int* status;
};

// dx_v = (1/T) [ g 1(v = target) + sum_j gt_j 1(v = id_j)
//                - p_v (g + sum gt + h (log p_v + H)) ]
// Bound by memory: 4096 x 131072 BF16 takes 321 us, 6.7 TB/s read and written.
// One pass: p_v comes from the saved maximum and log S, so a logit is read once and its
// gradient written once. The few columns that a token or an alternative names are written
// a second time, complete, by the CTA that owns them; their logits are read before
// anything is written, so `out` may be the logits' own buffer.
// p_v comes from log S in FP32, so a row's p share a factor that is off by half an ulp of log S
// (5e-7 near 10); the three numbers that the forward call saves a row hold no more.
// kVector: logits and gradient rows share their place within 16 bytes and go in 16-byte
// pieces; otherwise one value at a time, in 3.3 times the time for BF16 (4096 x 32000: 265 us, 81
// in pieces) and 2.2 for FP32 (509 x 32003 in rows of 32064, result packed: 42 us, 19).
template <typename T, bool kVector>
__global__ void __launch_bounds__(kThreads)
logprob_grad_kernel(const GradParams p) {
  constexpr int kN = Vec<T>::kN;
  constexpr int kUnroll = 4;
  __shared__ int64_t special[kMaxTop + 1];
  __shared__ float weight[kMaxTop + 1];
  grid_dependency_wait();
  grid_launch_dependents();
  const int tid = threadIdx.x;
  const int64_t row_id = blockIdx.x / static_cast<unsigned>(p.parts);
  const int part = static_cast<int>(blockIdx.x % static_cast<unsigned>(p.parts));
  // no __restrict__, plain loads: the two may be the same buffer
  const T* row = static_cast<const T*>(p.logits) + row_id * p.ld;
  T* out = static_cast<T*>(p.out) + row_id * p.out_ld;
  RowShape shape = row_shape(row, p.vocab);
  if (!kVector) shape = RowShape{0, 0, p.vocab};
  // parts past the row's last vector are empty; the last one holds the single values there
  const int64_t v0 = part * p.per_cta < shape.nv ? part * p.per_cta : shape.nv;
  const int64_t v1 = v0 + p.per_cta < shape.nv ? v0 + p.per_cta : shape.nv;
  const bool first = part == 0, last = part == p.parts - 1;

  const float m = p.stats[2 * row_id], log_s = p.stats[2 * row_id + 1];
  const float ent = p.entropy[row_id];
  const float h = p.g_entropy ? p.g_entropy[row_id] : 0.f;
  const int64_t target = p.targets[row_id];
  const bool empty = m == -kInf;
  const float sub = empty ? 0.f : m;
  const float nan = __uint_as_float(0x7FC00000u);
  const float g = target < 0 || empty ? 0.f : target >= p.vocab ? nan : p.g_logprob[row_id];
  bool bad = target >= p.vocab;
  float mass = g;
  for (int j = 0; j < p.top; ++j) {
    const int64_t id = p.top_id[row_id * p.top + j];
    if (id >= p.vocab) bad = true;
    else if (id >= 0) mass += p.g_top[row_id * p.top + j];
  }
  if (bad) {  // no column takes such a token's share: the row has no gradient
    mass = nan;
    if (first && tid == 0) latch_error(p.status, MXFP8_ERR_BAD_TARGET);
  }
  const float c = p.inv_t * kLog2e, base = log_s * kLog2e;
  // dx = -p (A + B t) / T + the named columns, t = log2 p. p is taken as 2^(t + 24) with
  // 2^-24 in A and B, since ex2 flushes subnormal results: so p is good down to 2^-150.
  constexpr float kLift = 24.f, kDrop = 0x1p-24f;
  // An empty row's gradient is zero even where h or a weight is not finite.
  const float A = empty ? 0.f : -(mass + h * ent) * p.inv_t * kDrop;
  const float B = empty ? 0.f : -h * kLn2 * p.inv_t * kDrop;
  auto grad_of = [&](float x) {
    const float t = max_nan((x - sub) * c - base, kLowest);
    return ex2(t + kLift) * fmaf(B, t, A);
  };

  // the columns named by the token and the alternatives, where this CTA owns them
  const int n_special = 1 + p.top;
  if (tid < n_special) {
    int64_t id = tid == 0 ? target : p.top_id[row_id * p.top + tid - 1];
    if (id >= p.vocab || id < 0) id = -1;
    special[tid] = id;
    weight[tid] = id < 0 ? 0.f : tid == 0 ? g : p.g_top[row_id * p.top + tid - 1];
  }
  __syncthreads();
  float fix = 0.f;
  int64_t fix_at = -1;
  if (tid < n_special && special[tid] >= 0 && !empty) {
    const int64_t id = special[tid];
    const int64_t lo = first ? 0 : shape.head + v0 * (kVector ? kN : 1);
    const int64_t hi = last ? p.vocab : shape.head + v1 * (kVector ? kN : 1);
    bool leads = id >= lo && id < hi;
    float w = 0.f;
    for (int j = 0; j < n_special; ++j) {
      if (special[j] != id) continue;
      if (j < tid) leads = false;  // the first that names a column writes it
      w += weight[j];
    }
    if (leads) {
      fix_at = id;
      fix = fmaf(w, p.inv_t, grad_of(Vec<T>::load(row + id)));
    }
  }
  __syncthreads();

  if constexpr (kVector) {
    const uint4* body = reinterpret_cast<const uint4*>(row + shape.head);
    uint4* obody = reinterpret_cast<uint4*>(out + shape.head);
    for (int64_t b = v0; b < v1; b += kUnroll * kThreads) {
      uint4 w[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int64_t v = b + u * kThreads + tid;
        w[u] = v < v1 ? body[v] : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int64_t v = b + u * kThreads + tid;
        float x[kN];
        Vec<T>::unpack(w[u], x);
#pragma unroll
        for (int i = 0; i < kN; ++i) x[i] = grad_of(x[i]);
        if (v < v1) obody[v] = Vec<T>::pack(x);
      }
    }
    const int64_t tail0 = shape.head + shape.nv * kN;
    if (first && tid < shape.head) Vec<T>::store(out + tid, grad_of(Vec<T>::load(row + tid)));
    if (last && tid < shape.tail)
      Vec<T>::store(out + tail0 + tid, grad_of(Vec<T>::load(row + tail0 + tid)));
  } else {
    for (int64_t v = v0 + tid; v < v1; v += kThreads)
      Vec<T>::store(out + v, grad_of(Vec<T>::load(row + v)));
  }
  __syncthreads();
  if (fix_at >= 0) Vec<T>::store(out + fix_at, fix);
}

template <typename... KArgs, typename... Args>
cudaError_t launch(void (*k)(KArgs...), unsigned grid, int threads, int cluster, bool early,
                   cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  cfg.attrs = attr;
  cfg.numAttrs = early ? pdl_attr(&attr[0]) : 0;
  if (cluster > 1) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attr[cfg.numAttrs].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[cfg.numAttrs].val.clusterDim.y = 1;
    attr[cfg.numAttrs].val.clusterDim.z = 1;
    ++cfg.numAttrs;
  }
  return cudaLaunchKernelEx(&cfg, k, args...);
}

// Threads of a CTA: few enough that each has 16 vectors or more of its part to stream, because
// the joins and the ranking after the stream are hidden only by other CTAs on the SM (4096 x
// 8000 BF16, top 8: 45 us with 256 threads, 30 with 128, 25 with 64; 2000 x 16000: 29, 23, 27;
// 4096 x 131072, top 32: 206, 231, 356); more where the rows alone would leave SMs short of
// threads.
template <typename T, bool kTop>
cudaError_t launch_forward(const Params& p, int split, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>(p.rows * split);
  const int64_t vectors = p.vocab / Vec<T>::kN / split;
  int threads = vectors >= 4096 ? 256 : vectors >= 1536 ? 128 : 64;
  while (threads < 256 && p.rows * split * threads < int64_t{1024} * num_sms()) threads *= 2;
  auto k = threads == 256   ? logprob_kernel<T, kTop, 256>
           : threads == 128 ? logprob_kernel<T, kTop, 128>
                            : logprob_kernel<T, kTop, 64>;
  // Up to two CTAs an SM may take their places while the kernel before still runs, which saves
  // 0.6 us (of 1 x 131072). Of more, some SMs would get two fewer than others
  // that way: 500 x 131072 BF16, top 5: 34 us, 38 with early places; 400 x 32000: 12.4 and 15.4.
  const bool early = grid <= 2u * static_cast<unsigned>(num_sms());
  return launch(k, grid, threads, split, early, stream, p, split);
}

}  // namespace

cudaError_t launch_logprob(const LogprobArgs& a, cudaStream_t stream) {
  if (a.rows == 0) return cudaSuccess;
  Params p{a.logits, a.rows, a.vocab, a.ld, a.targets, a.inv_t, a.logprob, a.entropy,
           a.stats, a.top, a.top_logprob, a.top_id, a.status};
  // CTAs per row: one for each SM while a part keeps 2048 values, two while it keeps 4096
  // 16-byte vectors, 16 a thread (top 5: 253 x 50021 FP32 takes 11% less in halves than whole;
  // 128 x 32000 BF16 12% more in quarters than in halves)
  const int64_t per_vector = a.fp32 ? 4 : 8;
  int split = 1;
  while (split < kMaxSplit && a.vocab >= 4096 * split &&
         (a.rows * split < num_sms() ||
          (a.rows * split < 2 * num_sms() && a.vocab / per_vector >= 8192 * split)))
    split *= 2;
  const int64_t grid = a.rows * split;
  if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
  return a.fp32 ? (a.top ? launch_forward<float, true>(p, split, stream)
                         : launch_forward<float, false>(p, split, stream))
                : (a.top ? launch_forward<__nv_bfloat16, true>(p, split, stream)
                         : launch_forward<__nv_bfloat16, false>(p, split, stream));
}

cudaError_t launch_logprob_grad(const LogprobGradArgs& a, cudaStream_t stream) {
  if (a.rows == 0) return cudaSuccess;
  GradParams p{a.logits, a.rows, a.vocab, a.ld, a.targets, a.inv_t, a.stats, a.entropy,
               a.g_logprob, a.g_entropy, a.top, a.top_id, a.g_top, a.out, a.out_ld, 0, 0,
               a.status};
  const int64_t size = a.fp32 ? 4 : 2;
  // the 16-byte path needs every row of both to start at the same place within 16 bytes
  const bool vector = ((reinterpret_cast<uintptr_t>(a.logits) ^
                        reinterpret_cast<uintptr_t>(a.out)) & 15u) == 0 &&
                      ((a.ld - a.out_ld) * size) % 16 == 0;
  const int64_t units = vector ? a.vocab / (16 / size) : a.vocab;  // bound on a row's vectors
  // parts of at least 4 vectors a thread, until the SMs are filled
  int64_t parts = 1;
  while (a.rows * parts < 8 * num_sms() && units / (2 * parts) >= 4 * kThreads) parts *= 2;
  p.parts = static_cast<int>(parts);
  p.per_cta = (units + parts - 1) / parts;
  if (p.per_cta < 1) p.per_cta = 1;
  const int64_t grid = a.rows * parts;
  if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
  auto k = a.fp32 ? (vector ? logprob_grad_kernel<float, true> : logprob_grad_kernel<float, false>)
                  : (vector ? logprob_grad_kernel<__nv_bfloat16, true>
                            : logprob_grad_kernel<__nv_bfloat16, false>);
  return launch(k, static_cast<unsigned>(grid), kThreads, 1, true, stream, p);
}

}  // namespace mxfp8
