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
// from a large logit. Sums, maxima and statistics are FP32 (per thread over a few hundred
// values, then joined pairwise); powers are taken in base 2 (one multiplication by
// log2(e) / T, then ex2).
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

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
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

  template <int kN>
  __device__ __forceinline__ void add(const float (&x)[kN], float c) {
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

struct Shared {
  float part[kWarps][3];
  float cta[3];                     // this CTA's m, S, E (read by the cluster's first CTA)
  float row[2];                     // the row's maximum and log S
  alignas(16) float thread_max[kThreads];  // read four at a time
  int chosen[kThreads];             // threads whose values may hold alternatives
  int num_chosen;
  uint32_t bar;                     // order of the smallest chosen thread maximum
  uint64_t keys[kMaxSplit * kMaxTop];
  uint64_t top[kMaxTop];            // this CTA's k best keys
};

// Keys [0, n) in sh.keys: the k largest, in order, into `out` (kNoKey where fewer exist).
__device__ __forceinline__ void rank_keys(const uint64_t* keys, int n, int k, uint64_t* out,
                                          int tid) {
  if (tid < k) out[tid] = kNoKey;
  __syncthreads();
  if (tid < n) {
    const uint64_t mine = keys[tid];
    int above = 0;
    for (int i = 0; i < n; ++i) above += keys[i] > mine;
    if (mine > kNoKey && above < k) out[above] = mine;
  }
  __syncthreads();
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

// One cluster of `split` CTAs per row; each CTA streams a contiguous part of it once.
//
// Bound by memory (2 or 4 bytes a logit). The alternatives do not slow the stream down: it
// only keeps each thread's maximum, which the softmax needs anyway. A value among the k
// largest sits in a thread whose maximum is among the k largest thread maxima, so only
// those threads' values, k / 256 of the row, are read again (from L2) and sorted into
// per-warp lists. Rows are split over a cluster only when there are too few of them to
// fill the GPU; the parts are joined through distributed shared memory, without a
// workspace.
template <typename T>
__global__ void __launch_bounds__(kThreads)
logprob_kernel(const Params p, int split) {
  constexpr int kN = Vec<T>::kN;
  constexpr int kUnroll = 4;
  __shared__ Shared sh;
  grid_dependency_wait();
  grid_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row_id = blockIdx.x / static_cast<unsigned>(split);
  const int rank = static_cast<int>(blockIdx.x % static_cast<unsigned>(split));
  const T* row = static_cast<const T*>(p.logits) + row_id * p.ld;
  const RowShape shape = row_shape(row, p.vocab);
  const int64_t v0 = shape.nv * rank / split, v1 = shape.nv * (rank + 1) / split;
  const uint4* body = reinterpret_cast<const uint4*>(row + shape.head);
  const bool has_head = rank == 0 && tid < shape.head;
  const bool has_tail = rank == split - 1 && tid < shape.tail;
  const int64_t tail0 = shape.head + shape.nv * kN;
  const float c = p.inv_t * kLog2e;

  Softmax sm;
  int64_t v = v0 + tid;
  for (; v + (kUnroll - 1) * kThreads < v1; v += kUnroll * kThreads) {
    uint4 w[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) w[u] = ld_nc_v4(body + v + u * kThreads);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      float x[kN];
      Vec<T>::unpack(w[u], x);
      sm.add(x, c);
    }
  }
  for (; v < v1; v += kThreads) {
    float x[kN];
    Vec<T>::unpack(ld_nc_v4(body + v), x);
    sm.add(x, c);
  }
  if (has_head || has_tail) {
    const float x[2] = {has_head ? Vec<T>::load(row + tid) : -kInf,
                        has_tail ? Vec<T>::load(row + tail0 + tid) : -kInf};
    sm.add(x, c);
  }
  const float own_max = sm.m;

  // join the CTA's threads
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float om = __shfl_xor_sync(0xFFFFFFFFu, sm.m, o);
    const float os = __shfl_xor_sync(0xFFFFFFFFu, sm.s, o);
    const float oe = __shfl_xor_sync(0xFFFFFFFFu, sm.e, o);
    sm.join(om, os, oe, c);
  }
  if (lane == 0) {
    sh.part[warp][0] = sm.m;
    sh.part[warp][1] = sm.s;
    sh.part[warp][2] = sm.e;
  }
  sh.thread_max[tid] = own_max;
  if (tid == 0) {
    sh.num_chosen = 0;
    sh.bar = 0xFFFFFFFFu;
  }
  __syncthreads();
  if (tid == 0) {
    Softmax all;
    for (int w = 0; w < kWarps; ++w) all.join(sh.part[w][0], sh.part[w][1], sh.part[w][2], c);
    sh.cta[0] = all.m;
    sh.cta[1] = all.s;
    sh.cta[2] = all.e;
  }

  if (p.top > 0) {
    // threads with fewer than k larger thread maxima
    int above = 0;
    for (int i = 0; i < kThreads; i += 4) {
      const float4 o = *reinterpret_cast<const float4*>(&sh.thread_max[i]);
      above += (o.x > own_max) + (o.y > own_max) + (o.z > own_max) + (o.w > own_max);
    }
    if (above < p.top && own_max > -kInf) {
      sh.chosen[atomicAdd(&sh.num_chosen, 1)] = tid;
      atomicMin(&sh.bar, order_of(own_max));
    }
    __syncthreads();
    WarpTop best;
    const int n = sh.num_chosen;
    // k chosen maxima bound the k-th best key from below; fewer do not
    best.least = n >= p.top ? (static_cast<uint64_t>(sh.bar) << 32) - 1 : kNoKey;
    const int64_t steps = (v1 - v0 + kThreads - 1) / kThreads;
    for (int q = warp; q < n; q += kWarps) {
      const int owner = sh.chosen[q];
      for (int64_t j0 = 0; j0 < steps; j0 += 32) {
        const int64_t at = v0 + owner + (j0 + lane) * kThreads;
        const bool live = at < v1;
        float x[kN];
        Vec<T>::unpack(live ? __ldg(body + at) : make_uint4(0, 0, 0, 0), x);
#pragma unroll
        for (int i = 0; i < kN; ++i)
          best.offer(live ? key_of(x[i], static_cast<uint32_t>(shape.head + at * kN + i)) : kNoKey,
                     p.top, lane);
      }
      // the owner's single values
      uint64_t key = kNoKey;
      if (lane == 0 && rank == 0 && owner < shape.head)
        key = key_of(Vec<T>::load(row + owner), static_cast<uint32_t>(owner));
      if (lane == 1 && rank == split - 1 && owner < shape.tail)
        key = key_of(Vec<T>::load(row + tail0 + owner), static_cast<uint32_t>(tail0 + owner));
      best.offer(key, p.top, lane);
    }
    sh.keys[warp * kMaxTop + lane] = lane < p.top ? best.mine : kNoKey;
    __syncthreads();
    rank_keys(sh.keys, kWarps * kMaxTop, p.top, sh.top, tid);
  } else {
    __syncthreads();
  }

  // join the cluster's CTAs in its first
  if (split > 1) {
    cluster_sync();
    if (rank == 0) {
      if (p.top > 0) {
        const int r = tid / kMaxTop, i = tid % kMaxTop;
        uint64_t key = kNoKey;
        if (r < split && i < p.top) {
          const uint32_t from = cluster_map(&sh.top[i], static_cast<uint32_t>(r));
          asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(key) : "r"(from) : "memory");
        }
        sh.keys[tid] = key;
      }
      if (tid == 0) {
        Softmax all;
        for (int r = 0; r < split; ++r) {
          float o[3];
          for (int i = 0; i < 3; ++i) {
            const uint32_t from = cluster_map(&sh.cta[i], static_cast<uint32_t>(r));
            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(o[i]) : "r"(from) : "memory");
          }
          all.join(o[0], o[1], o[2], c);
        }
        sh.part[0][0] = all.m;
        sh.part[0][1] = all.s;
        sh.part[0][2] = all.e;
      }
    }
    cluster_sync();  // no CTA leaves while its shared memory is being read
    if (rank != 0) return;
    if (tid == 0)
      for (int i = 0; i < 3; ++i) sh.cta[i] = sh.part[0][i];
    __syncthreads();
    if (p.top > 0) rank_keys(sh.keys, kThreads, p.top, sh.top, tid);
  }

  if (tid == 0) {
    const float m = sh.cta[0], s = sh.cta[1], e = sh.cta[2];
    const bool empty = m == -kInf && s == 0.f;  // every logit -inf (a NaN makes s NaN)
    const float log_s = empty ? 0.f : logf(s);
    const int64_t target = p.targets[row_id];
    float lp = 0.f;
    if (target >= p.vocab) {
      latch_error(p.status, MXFP8_ERR_BAD_TARGET);
      lp = __uint_as_float(0x7FC00000u);
    } else if (target >= 0) {
      lp = empty ? -kInf : (Vec<T>::load(row + target) - m) * p.inv_t - log_s;
    }
    if (isnan(s)) lp = s;
    p.logprob[row_id] = lp;
    p.entropy[row_id] = empty ? 0.f : log_s - kLn2 * e / s;
    p.stats[2 * row_id] = isnan(s) ? s : m;
    p.stats[2 * row_id + 1] = log_s;
    sh.row[0] = isnan(s) ? s : m;
    sh.row[1] = log_s;
  }
  if (p.top > 0) {
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
// One pass: p_v comes from the saved maximum and log S, so a logit is read once and its
// gradient written once. The few columns that a token or an alternative names are written
// a second time, complete, by the CTA that owns them; their logits are read before
// anything is written, so `out` may be the logits' own buffer.
// kVector: logits and gradient rows share their place within 16 bytes and go in 16-byte
// pieces; otherwise one value at a time.
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
  const bool bad = target >= p.vocab;
  if (bad && first && tid == 0) latch_error(p.status, MXFP8_ERR_BAD_TARGET);
  const float g = target < 0 || empty ? 0.f : bad ? __uint_as_float(0x7FC00000u)
                                                  : p.g_logprob[row_id];
  float mass = g;
  for (int j = 0; j < p.top; ++j) {
    const int64_t id = p.top_id[row_id * p.top + j];
    if (id >= 0) mass += p.g_top[row_id * p.top + j];
  }
  const float c = p.inv_t * kLog2e, base = log_s * kLog2e;
  // dx = -p (A + B t) / T + the named columns, t = log2 p. p is taken as 2^(t + 24) with
  // 2^-24 in A and B, since ex2 flushes subnormal results: so p is good down to 2^-150.
  constexpr float kLift = 24.f, kDrop = 0x1p-24f;
  const float A = -(mass + h * ent) * p.inv_t * kDrop, B = -h * kLn2 * p.inv_t * kDrop;
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
cudaError_t launch(void (*k)(KArgs...), unsigned grid, int cluster, cudaStream_t stream,
                   Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
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

}  // namespace

cudaError_t launch_logprob(const LogprobArgs& a, cudaStream_t stream) {
  if (a.rows == 0) return cudaSuccess;
  Params p{a.logits, a.rows, a.vocab, a.ld, a.targets, a.inv_t, a.logprob, a.entropy,
           a.stats, a.top, a.top_logprob, a.top_id, a.status};
  // CTAs per row: enough to fill the SMs, while each part keeps at least 2048 values
  int split = 1;
  while (split < kMaxSplit && a.rows * split < 2 * num_sms() && a.vocab >= 4096 * split)
    split *= 2;
  const int64_t grid = a.rows * split;
  if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
  return launch(a.fp32 ? logprob_kernel<float> : logprob_kernel<__nv_bfloat16>,
                static_cast<unsigned>(grid), split, stream, p, split);
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
  return launch(k, static_cast<unsigned>(grid), 1, stream, p);
}

}  // namespace mxfp8
