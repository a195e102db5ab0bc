// moe_route_kernels.cuh -- the router of a mixture-of-experts layer: the top-k choice of experts,
// its weights, the per-expert counts, the balance loss of each sequence, and their gradient.
//
// For a row of logits l (E experts), p = softmax(l).  The k largest logits are chosen (ties: the
// lowest expert first); a logit of -inf, or NaN, is never chosen, and a row without a choice (or
// with mask = 0) is not routed.  Over the n routed rows of a sequence:
//   f_e = count_e / sum(count),  P_e = mean of p_e,  loss = E * sum_e f_e P_e,
//   slope_e = d loss / d p_te = E f_e / n   (the counts are not differentiated).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>
#include <cstring>

#include "cluster_ptx.cuh"
#include "sm100_ptx.cuh"

namespace fg {

constexpr int kRouteThreads = 256;
constexpr int kRouteWarps = kRouteThreads / 32;
constexpr int kRouteMaxK = 32;
constexpr int kRouteMaxCluster = 8;

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <typename T>
struct IsHalf {
  static constexpr bool value = false;
};
template <>
struct IsHalf<__half> {
  static constexpr bool value = true;
};
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// Orders a row's choices: a larger key is an earlier choice.  The upper part is the logit's fp32 bits made
// monotonic, the lower ten bits count columns down, so that equal logits come lowest expert first.  bf16
// and fp16 values have no fp32 bits below the 13th, so the key is one 32-bit word, which one warp
// reduction orders; fp32 logits take 64 bits and two reductions.  -0 and +0 are equal; -inf and NaN,
// which are never chosen, have keys below kClosed.
template <typename T>
struct RouteKey {
  typedef uint32_t type;
  static constexpr type kClosed = 0x00800000u;  // keys of -inf: 0x007FFC00 + column
  static __device__ __forceinline__ type make(float v, int inverse_col) {
    const uint32_t u = __float_as_uint(fmaxf(v + 0.0f, -INFINITY));
    return ((u ^ (static_cast<uint32_t>(static_cast<int>(u) >> 31) | 0x80000000u)) & 0xFFFFFC00u) |
           static_cast<uint32_t>(inverse_col);
  }
  static __device__ __forceinline__ int col(type k) { return 1023 - static_cast<int>(k & 1023u); }
  static __device__ __forceinline__ float logit(type k) {
    const uint32_t u = k & 0xFFFFFC00u;
    return __uint_as_float((u & 0x80000000u) ? (u & 0x7FFFFFFFu) : ~u & 0xFFFFFC00u);
  }
};
template <>
struct RouteKey<float> {
  typedef unsigned long long type;
  static constexpr type kClosed = 0x0080000000000000ull;
  static __device__ __forceinline__ type make(float v, int inverse_col) {
    const uint32_t u = __float_as_uint(fmaxf(v + 0.0f, -INFINITY));
    const uint32_t key = u ^ (static_cast<uint32_t>(static_cast<int>(u) >> 31) | 0x80000000u);
    return (static_cast<type>(key) << 32) | static_cast<uint32_t>(inverse_col);
  }
  static __device__ __forceinline__ int col(type k) { return 1023 - static_cast<int>(k & 1023u); }
  static __device__ __forceinline__ float logit(type k) {
    const uint32_t u = static_cast<uint32_t>(k >> 32);
    return __uint_as_float((u & 0x80000000u) ? (u & 0x7FFFFFFFu) : ~u);
  }
};

// e^(x - high), high the row's largest logit.  The difference is formed first: with the type's lowest
// value in every place of a row, a product with log2(e) before it would overflow.  expf, not ex2 of the rounded
// product: that would lose as many units in the last place as x lies below high, and all below 2^-126.
__device__ __forceinline__ float softmax_exp(float x, float high) { return expf(x - high); }

// Reductions over the LPR lanes that hold one row (LPR a power of two).
template <int LPR, int N>
__device__ __forceinline__ void row_sums(float (&v)[N]) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
}
template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
  float v[1] = {x};
  row_sums<LPR>(v);
  return v[0];
}
template <int LPR>
__device__ __forceinline__ float row_max(float v) {
  if constexpr (LPR == 32) {  // one integer reduction of the bits made monotonic
    const uint32_t u = __float_as_uint(v);
    const uint32_t top = __reduce_max_sync(0xffffffffu, u ^ (static_cast<uint32_t>(static_cast<int>(u) >> 31) | 0x80000000u));
    return __uint_as_float((top & 0x80000000u) ? (top & 0x7FFFFFFFu) : ~top);
  } else {
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
  }
}
template <int LPR>
__device__ __forceinline__ uint32_t row_best(uint32_t v) {
  if constexpr (LPR == 32) {
    return __reduce_max_sync(0xffffffffu, v);
  } else {
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
  }
}
template <int LPR>
__device__ __forceinline__ unsigned long long row_best(unsigned long long v) {
  if constexpr (LPR == 32) {
    const uint32_t hi = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(v >> 32));
    const uint32_t lo = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(v >> 32) == hi ? static_cast<uint32_t>(v) : 0u);
    return (static_cast<unsigned long long>(hi) << 32) | lo;
  } else {
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) {
      const unsigned long long w = __shfl_xor_sync(0xffffffffu, v, o);
      if (w > v) v = w;
    }
    return v;
  }
}

// Batcher's odd-even merge sort of registers, largest first: sort_falling sorts v[LO .. LO + N), merge_falling merges
// the sorted halves of its elements LO, LO + STEP, ...
template <int A, int B, typename K, int M>
__device__ __forceinline__ void order_falling(K (&v)[M]) {
  const K a = v[A], b = v[B];
  v[A] = a > b ? a : b;
  v[B] = a > b ? b : a;
}
template <int LO, int END, int STEP, typename K, int M>
__device__ __forceinline__ void order_pairs(K (&v)[M]) {
  if constexpr (LO + STEP < END) {
    order_falling<LO, LO + STEP>(v);
    order_pairs<LO + 2 * STEP, END, STEP>(v);
  }
}
template <int LO, int N, int STEP, typename K, int M>
__device__ __forceinline__ void merge_falling(K (&v)[M]) {
  if constexpr (2 * STEP < N) {
    merge_falling<LO, N, 2 * STEP>(v);
    merge_falling<LO + STEP, N, 2 * STEP>(v);
    order_pairs<LO + STEP, LO + N, STEP>(v);
  } else {
    order_falling<LO, LO + STEP>(v);
  }
}
template <int LO, int N, typename K, int M>
__device__ __forceinline__ void sort_falling(K (&v)[M]) {
  if constexpr (N > 1) {
    sort_falling<LO, N / 2>(v);
    sort_falling<LO + N / 2, N / 2>(v);
    merge_falling<LO, N, 1>(v);
  }
}

// Value i of lane `sub` of a row is column (i / V * LPR + sub) * V + i % V: V consecutive columns
// per load, the lanes side by side.
template <int LPR, int V>
__device__ __forceinline__ int route_col(int i, int sub) {
  return (i / V * LPR + sub) * V + i % V;
}

// One row's values of this lane, as they are; columns at or past E read as -inf.  V > 1: E % V == 0
// and the rows 16-byte aligned (V * sizeof(T) == 16).
template <typename T, int LPR, int NPL, int V>
__device__ __forceinline__ void load_logits(const T* row, int E, int sub, T (&x)[NPL]) {
#pragma unroll
  for (int i = 0; i < NPL; i += V) {
    const int c = route_col<LPR, V>(i, sub);
    if constexpr (V == 1) {
      x[i] = c < E ? row[c] : from_f32<T>(-INFINITY);
    } else {
      uint4 raw;
      if (c < E) {
        raw = *reinterpret_cast<const uint4*>(row + c);
      } else {
        const uint32_t none = sizeof(T) == 4 ? 0xFF800000u : IsHalf<T>::value ? 0xFC00FC00u : 0xFF80FF80u;
        raw = make_uint4(none, none, none, none);
      }
      memcpy(&x[i], &raw, 16);
    }
  }
}

struct RouteParams {
  const void* logits;   // [S][T][E]
  const uint8_t* mask;  // [S][T], nullptr: every row
  int* ids;             // [S][T][k]
  float* weights;       // [S][T][k]
  int* counts;          // [S][E]
  float* loss;          // [S]
  float* slope;         // [S][E]
  float* part_p;        // [S][chunks][E]: sums of p over a chunk's rows
  int* part_n;          // [S][chunks][E + 1]: counts of a chunk, then its routed rows
  int T, E, k, chunks, rows_per_chunk, renorm;
};

// What the sums over a sequence give.  Called by all threads of one CTA; thread e < E holds column e's
// sum of p and count; rows: the routed tokens (same in every thread).
__device__ __forceinline__ void route_finish(const RouteParams& p, int seq, float sum, int n, int rows, float* s_red,
                                             uint32_t* s_total) {
  const int e = threadIdx.x, warps = blockDim.x / 32;
  // all choices of the sequence, T k of them, may pass 2^32: the halves of the counts are summed apart, in 32 bits each
  const uint32_t mine = e < p.E ? n : 0;
  const uint32_t low = __reduce_add_sync(0xffffffffu, mine & 0xffffu), high = __reduce_add_sync(0xffffffffu, mine >> 16);
  if (e < 2) s_total[e] = 0;
  __syncthreads();
  if ((e & 31) == 0) {
    if (low) atomicAdd(&s_total[0], low);
    if (high) atomicAdd(&s_total[1], high);
  }
  __syncthreads();
  const unsigned long long choices = (static_cast<unsigned long long>(s_total[1]) << 16) + s_total[0];
  const float total = static_cast<float>(max(choices, 1ull)) * static_cast<float>(max(rows, 1));
  const float slope = static_cast<float>(p.E) * static_cast<float>(n) / total;
  if (e < p.E) {
    p.counts[static_cast<size_t>(seq) * p.E + e] = n;
    p.slope[static_cast<size_t>(seq) * p.E + e] = slope;
  }
  float v = row_sum<32>(e < p.E ? slope * sum : 0.0f);
  if ((e & 31) == 0) s_red[e >> 5] = v;
  __syncthreads();
  if (e < 32) {
    v = row_sum<32>(e < warps ? s_red[e] : 0.0f);
    if (e == 0) p.loss[seq] = v;
  }
}

// Forward, one CTA per (chunk of rows, sequence).  LPR lanes hold a row, NPL values each, so a warp
// works on 32 / LPR rows at once; the next rows are loaded while the present ones are worked on.  Each
// lane sorts its keys once (a network in registers), then every choice is one reduction over the heads of
// the lanes' lists and a shift in the winner's.  Bound by the integer pipe, about 510 instructions per row of
// 256: 32768 rows in 8 sequences, bf16, top 8, in 26 us with the finishing kernel (17 MB, which take 2.6).
// CLUSTER: the sequence's CTAs are one cluster, whose first CTA sums the others' parts over distributed
// shared memory and finishes; otherwise the parts go to memory for moe_route_finish_kernel.
template <typename T, int LPR, int NPL, int V, bool CLUSTER>
__global__ void __launch_bounds__(kRouteThreads) moe_route_kernel(const RouteParams p) {
  typedef RouteKey<T> Key;
  typedef typename Key::type K;
  constexpr int RPW = 32 / LPR;
  constexpr int EP = LPR * NPL;
  __shared__ int s_cnt[EP + 1];
  __shared__ float s_sum[kRouteWarps][EP];
  __shared__ K s_key[kRouteWarps][RPW][kRouteMaxK];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane % LPR, rw = lane / LPR;
  const int seq = blockIdx.y, chunk = blockIdx.x;
  for (int i = threadIdx.x; i <= EP; i += kRouteThreads) s_cnt[i] = 0;
  __syncthreads();
  pdl_wait_prior_grid();
  pdl_launch_dependents();

  float acc[NPL];
#pragma unroll
  for (int i = 0; i < NPL; ++i) acc[i] = 0.0f;
  // rows are counted from the chunk's first one, so that row numbers next to 2^31 do not overflow
  const int first = chunk * p.rows_per_chunk, last = min(p.T - first, p.rows_per_chunk);
  const size_t base = static_cast<size_t>(seq) * p.T + first;
  const T* logits = static_cast<const T*>(p.logits) + base * p.E;
  const uint8_t* mask = p.mask ? p.mask + base : nullptr;
  int* ids = p.ids + base * p.k;
  float* weights = p.weights + base * p.k;
  T next[NPL];
  bool next_live = false;
  auto fetch = [&](int r0) {  // rows behind the last one repeat it and are dropped later
    const int r = min(r0 + rw, last - 1);
    next_live = !mask || mask[r];
    load_logits<T, LPR, NPL, V>(logits + static_cast<size_t>(r) * p.E, p.E, sub, next);
  };
  K* keys = s_key[warp][rw];
  int r0 = warp * RPW;
  if (r0 < last) fetch(r0);
  for (; r0 < last; r0 += kRouteWarps * RPW) {
    const int r = r0 + rw;
    const bool live = r < last && next_live;
    if (__ballot_sync(0xffffffffu, live) == 0) {  // all of the warp's rows are masked
      if (r < last) {
        for (int j = sub; j < p.k; j += LPR) {
          ids[static_cast<size_t>(r) * p.k + j] = -1;
          weights[static_cast<size_t>(r) * p.k + j] = 0.0f;
        }
      }
      if (r0 + kRouteWarps * RPW < last) fetch(r0 + kRouteWarps * RPW);
      continue;
    }
    float x[NPL];
    K key[NPL];
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      x[i] = to_f32(next[i]);
      key[i] = Key::make(x[i], 1023 - route_col<LPR, V>(i, sub));
    }
    if (r0 + kRouteWarps * RPW < last) fetch(r0 + kRouteWarps * RPW);
    sort_falling<0, NPL>(key);
    K best = row_best<LPR>(key[0]);
    const bool routed = live && best >= Key::kClosed;
    const float high = routed ? Key::logit(best) : 0.0f;
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      x[i] = softmax_exp(x[i], high);
      sum += x[i];
    }
    // the winner's lane records the choice and moves its list on (keys differ by their columns; 0 once a list
    // is empty).  Up to eight choices, the common case: only as much of a list is moved as is still needed.
    if (p.k <= 8) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (j >= p.k) break;
        const bool wins = key[0] == best;
        if (wins) keys[j] = best;
#pragma unroll
        for (int i = 0; i < (NPL < 7 - j ? NPL : 7 - j); ++i) key[i] = wins ? (i + 1 < NPL ? key[i + 1] : K(0)) : key[i];
        best = row_best<LPR>(key[0]);
      }
    } else {
      for (int j = 0; j < p.k; ++j) {
        if (key[0] == best) {
          keys[j] = best;
#pragma unroll
          for (int i = 0; i < NPL; ++i) key[i] = i + 1 < NPL ? key[i + 1] : K(0);
        }
        best = row_best<LPR>(key[0]);
      }
    }
    __syncwarp();
    float sums[2] = {sum, 0.0f};  // over all columns; over the choices
    K choice = 0;
    if (sub < p.k && routed) choice = keys[sub];
    float u = choice >= Key::kClosed ? softmax_exp(Key::logit(choice), high) : 0.0f;
    sums[1] = u;
    if constexpr (LPR < kRouteMaxK) {
      if (routed)
        for (int j = sub + LPR; j < p.k; j += LPR)
          if (keys[j] >= Key::kClosed) sums[1] += softmax_exp(Key::logit(keys[j]), high);
    }
    row_sums<LPR>(sums);
    const float inv = 1.0f / sums[0];
    if (routed) {
#pragma unroll
      for (int i = 0; i < NPL; ++i) acc[i] = fmaf(x[i], inv, acc[i]);
    }
    if (r < last) {
      const float scale = p.renorm ? 1.0f / sums[1] : inv;
      auto put = [&](int j, K c, float w) {
        const bool chosen = c >= Key::kClosed;
        const size_t at = static_cast<size_t>(r) * p.k + j;
        ids[at] = chosen ? Key::col(c) : -1;
        weights[at] = chosen ? w * scale : 0.0f;
        if (chosen) atomicAdd(&s_cnt[Key::col(c)], 1);
      };
      if (sub < p.k) put(sub, choice, u);
      if constexpr (LPR < kRouteMaxK) {
        for (int j = sub + LPR; j < p.k; j += LPR) {
          choice = routed ? keys[j] : K(0);
          put(j, choice, choice >= Key::kClosed ? softmax_exp(Key::logit(choice), high) : 0.0f);
        }
      }
      if (sub == 0 && routed) atomicAdd(&s_cnt[EP], 1);
    }
    __syncwarp();
  }
  // sums of p over the CTA's rows in a fixed order: the rows of a warp's lanes, then the warps
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
#pragma unroll
    for (int o = LPR; o < 32; o <<= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
    if (rw == 0) s_sum[warp][route_col<LPR, V>(i, sub)] = acc[i];
  }
  __syncthreads();
  const size_t slot = static_cast<size_t>(seq) * p.chunks + chunk;
  for (int e = threadIdx.x; e < p.E; e += kRouteThreads) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kRouteWarps; ++w) v += s_sum[w][e];
    if constexpr (CLUSTER) {
      s_sum[0][e] = v;
    } else {
      p.part_p[slot * p.E + e] = v;
      p.part_n[slot * (p.E + 1) + e] = s_cnt[e];
    }
  }
  if constexpr (CLUSTER) {
    __shared__ float s_red[kRouteWarps];
    __shared__ uint32_t s_total[2];
    cluster_sync_all();
    if (chunk == 0) {
      static_assert(EP <= kRouteThreads, "one column per thread");
      float v = 0.0f;
      int n = 0, rows = 0;
      const int e = threadIdx.x;
      const uint32_t sum_at = smem_addr(&s_sum[0][min(e, EP - 1)]), n_at = smem_addr(&s_cnt[min(e, EP - 1)]),
                     rows_at = smem_addr(&s_cnt[EP]);
      for (int c = 0; c < p.chunks; ++c) {
        v += ld_dsmem_f32(mapa_shared(sum_at, c));
        n += __float_as_int(ld_dsmem_f32(mapa_shared(n_at, c)));
        rows += __float_as_int(ld_dsmem_f32(mapa_shared(rows_at, c)));
      }
      cluster_sync_all();  // the parts have been read
      route_finish(p, seq, v, n, rows, s_red, s_total);
    } else {
      cluster_sync_all();  // no CTA leaves before its part has been read
    }
  } else {
    if (threadIdx.x == 0) p.part_n[slot * (p.E + 1) + p.E] = s_cnt[EP];
  }
}

// Sums of the chunks of one sequence in a fixed order, then its counts, slopes and loss.  A cluster of
// kFinishCluster CTAs of 1024 threads: each takes as many parts of the chunks side by side as columns leave room
// for, and the first sums the CTAs' parts over distributed shared memory (the router of 32768 rows of 256 in one
// sequence: 29 us; at 586 chunks one CTA here took 9 us more than eight).
constexpr int kFinishCluster = 8;
__global__ void __launch_bounds__(1024) moe_route_finish_kernel(const RouteParams p) {
  __shared__ float s_part[1024];
  __shared__ int s_cnt[1024];
  __shared__ float s_red[32];
  __shared__ uint32_t s_total[2];
  __shared__ int s_rows;
  const int seq = blockIdx.y, rank = static_cast<int>(cluster_ctarank());
  if (threadIdx.x == 0) s_rows = 0;
  __syncthreads();
  pdl_wait_prior_grid();
  pdl_launch_dependents();
  const size_t slot = static_cast<size_t>(seq) * p.chunks;
  const int cols = (p.E + 31) / 32 * 32, parts = 1024 / cols;
  const int e = threadIdx.x % cols, part = threadIdx.x / cols;
  float sum = 0.0f;
  int n = 0;
  if (e < p.E && part < parts) {
#pragma unroll 8
    for (int c = rank * parts + part; c < p.chunks; c += kFinishCluster * parts) {
      sum += p.part_p[(slot + c) * p.E + e];
      n += p.part_n[(slot + c) * (p.E + 1) + e];
    }
  }
  s_part[threadIdx.x] = sum;
  s_cnt[threadIdx.x] = n;
  int rows = 0;
  for (int c = rank * 1024 + threadIdx.x; c < p.chunks; c += kFinishCluster * 1024)
    rows += p.part_n[(slot + c) * (p.E + 1) + p.E];
  if (rows) atomicAdd(&s_rows, rows);
  __syncthreads();
  if (part == 0) {
    for (int q = 1; q < parts; ++q) {
      sum += s_part[q * cols + e];
      n += s_cnt[q * cols + e];
    }
    s_part[e] = sum;
    s_cnt[e] = n;
  }
  cluster_sync_all();
  if (rank == 0) {
    sum = 0.0f;
    n = 0;
    rows = 0;
    const uint32_t sum_at = smem_addr(&s_part[e]), n_at = smem_addr(&s_cnt[e]), rows_at = smem_addr(&s_rows);
#pragma unroll
    for (int c = 0; c < kFinishCluster; ++c) {
      sum += ld_dsmem_f32(mapa_shared(sum_at, c));
      n += __float_as_int(ld_dsmem_f32(mapa_shared(n_at, c)));
      rows += __float_as_int(ld_dsmem_f32(mapa_shared(rows_at, c)));
    }
  }
  cluster_sync_all();  // the parts have been read
  if (rank != 0) return;
  // columns past E (and threads of other parts) hold nothing
  route_finish(p, seq, sum, threadIdx.x < p.E ? n : 0, rows, s_red, s_total);
}

struct RouteGradParams {
  const void* logits;         // [S][T][E]
  const int* ids;             // [S][T][k]
  const float* slope;         // [S][E]
  const float* grad_weights;  // [S][T][k] or nullptr
  const float* grad_loss;     // [S] or nullptr
  void* grad_logits;          // [S][T][E]
  int T, E, k, rows_per_chunk, renorm;
};

// Backward.  With u_e = e^(l_e - max), h_e = grad_loss * slope_e and g_j the gradient of weight j:
//   not renormalised:  d l_e = p_e (h_e - (sum u h + sum_j u_j g_j) / sum u)   (+ p_j g_j at the choices)
//   renormalised:      d l_e = p_e (h_e - sum u h / sum u)  (+ w_j (g_j - sum_j w g) at the choices),
// w the softmax over the chosen logits.  All four sums are reduced together.  Rows without a choice get
// zeros.  What the choices add goes through a row of shared memory, which is zero between rows.  32768 rows of
// 256, bf16, top 8: 15.8 us for 36 MB, bound by instructions (about 350 a row).
template <typename T, int LPR, int NPL, int V>
__global__ void __launch_bounds__(kRouteThreads) moe_route_backward_kernel(const RouteGradParams p) {
  constexpr int RPW = 32 / LPR;
  constexpr int EP = LPR * NPL;
  __shared__ __align__(16) float s_add[kRouteWarps][RPW][EP];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane % LPR, rw = lane / LPR;
  const int seq = blockIdx.y;
  for (int i = threadIdx.x; i < kRouteWarps * RPW * EP; i += kRouteThreads) (&s_add[0][0][0])[i] = 0.0f;
  __syncthreads();
  pdl_wait_prior_grid();
  pdl_launch_dependents();
  float* add = s_add[warp][rw];
  float h[NPL];
  const float g = p.grad_loss ? p.grad_loss[seq] : 0.0f;
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const int c = route_col<LPR, V>(i, sub);
    h[i] = p.grad_loss && c < p.E ? g * p.slope[static_cast<size_t>(seq) * p.E + c] : 0.0f;
  }
  // as in the forward kernel, rows from the chunk's first one
  const int first = blockIdx.x * p.rows_per_chunk, last = min(p.T - first, p.rows_per_chunk);
  const size_t base = static_cast<size_t>(seq) * p.T + first;
  const T* all = static_cast<const T*>(p.logits) + base * p.E;
  T* out_all = static_cast<T*>(p.grad_logits) + base * p.E;
  const int* ids = p.ids + base * p.k;
  const float* weights = p.grad_weights ? p.grad_weights + base * p.k : nullptr;
  T next[NPL];
  int next_id = -1;
  float next_g = 0.0f;
  auto choice = [&](int r, int j, int& id, float& gw) {
    const size_t at = static_cast<size_t>(r) * p.k + j;
    id = ids[at];
    if (static_cast<unsigned>(id) >= static_cast<unsigned>(p.E)) id = -1;
    gw = weights ? weights[at] : 0.0f;
  };
  auto fetch = [&](int r0) {
    const int r = min(r0 + rw, last - 1);
    load_logits<T, LPR, NPL, V>(all + static_cast<size_t>(r) * p.E, p.E, sub, next);
    if (sub < p.k) choice(r, sub, next_id, next_g);
  };
  int r0 = warp * RPW;
  if (r0 < last) fetch(r0);
  for (; r0 < last; r0 += kRouteWarps * RPW) {
    const int r = min(r0 + rw, last - 1);
    const T* logits = all + static_cast<size_t>(r) * p.E;
    float x[NPL];
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      x[i] = to_f32(next[i]);
      m = fmaxf(m, x[i]);
    }
    const int id = next_id;
    const float gw = next_g;
    if (r0 + kRouteWarps * RPW < last) fetch(r0 + kRouteWarps * RPW);
    bool any = id >= 0;
    if constexpr (LPR < kRouteMaxK) {
      for (int j = sub + LPR; j < p.k; j += LPR) any |= static_cast<unsigned>(ids[static_cast<size_t>(r) * p.k + j]) < static_cast<unsigned>(p.E);
    }
    const uint32_t votes = __ballot_sync(0xffffffffu, any);
    const bool routed = (votes >> (rw * LPR)) & (LPR == 32 ? 0xffffffffu : (1u << (LPR & 31)) - 1);
    T* out = out_all + static_cast<size_t>(r) * p.E;
    const bool write = r0 + rw < last;
    if (votes == 0) {  // none of the warp's rows was routed
#pragma unroll
      for (int i = 0; i < NPL; i += V) {
        const int c = route_col<LPR, V>(i, sub);
        if (c >= p.E || !write) continue;
        if constexpr (V == 1)
          out[c] = from_f32<T>(0.0f);
        else
          *reinterpret_cast<uint4*>(out + c) = make_uint4(0u, 0u, 0u, 0u);
      }
      continue;
    }
    const float chosen = id >= 0 ? to_f32(logits[id]) : 0.0f;  // the row's own: in L1
    const float high = row_max<LPR>(m);
    // sums of u, of u h, of u over the choices, of u g over the choices
    float sums[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      x[i] = softmax_exp(x[i], high);
      sums[0] += x[i];
      sums[1] = fmaf(x[i], h[i], sums[1]);
    }
    const float u = id >= 0 ? softmax_exp(chosen, high) : 0.0f;
    sums[2] = u;
    sums[3] = id >= 0 ? u * gw : 0.0f;
    if constexpr (LPR < kRouteMaxK) {
      for (int j = sub + LPR; j < p.k; j += LPR) {
        int id2;
        float gw2;
        choice(r, j, id2, gw2);
        if (id2 < 0) continue;
        const float u2 = softmax_exp(to_f32(logits[id2]), high);
        sums[2] += u2;
        sums[3] = fmaf(u2, gw2, sums[3]);
      }
    }
    row_sums<LPR>(sums);
    const float inv = 1.0f / sums[0];
    const float top = p.renorm ? 1.0f / sums[2] : inv;
    const float mean = p.renorm ? sums[3] * top : 0.0f;
    const float dot = (p.renorm ? sums[1] : sums[1] + sums[3]) * inv;
    if (weights) {  // shared atomics: a choice may stand twice
      if (id >= 0) atomicAdd(&add[id], u * top * (gw - mean));
      if constexpr (LPR < kRouteMaxK) {
        for (int j = sub + LPR; j < p.k; j += LPR) {
          int id2;
          float gw2;
          choice(r, j, id2, gw2);
          if (id2 >= 0) atomicAdd(&add[id2], softmax_exp(to_f32(logits[id2]), high) * top * (gw2 - mean));
        }
      }
      __syncwarp();
    }
#pragma unroll
    for (int i = 0; i < NPL; i += V) {
      const int c = route_col<LPR, V>(i, sub);
      alignas(16) T t[V];
      alignas(16) float a[V];
      if constexpr (V % 4 == 0) {
#pragma unroll
        for (int v = 0; v < V; v += 4) *reinterpret_cast<float4*>(a + v) = *reinterpret_cast<const float4*>(add + c + v);
      } else {
        a[0] = add[c];
      }
#pragma unroll
      for (int v = 0; v < V; ++v) t[v] = from_f32<T>(routed ? fmaf(x[i + v] * inv, h[i + v] - dot, a[v]) : 0.0f);
      if (c < p.E && write) {
        if constexpr (V == 1)
          out[c] = t[0];
        else
          *reinterpret_cast<uint4*>(out + c) = *reinterpret_cast<const uint4*>(t);
      }
    }
    if (weights) {
      __syncwarp();
      if (id >= 0) add[id] = 0.0f;
      if constexpr (LPR < kRouteMaxK) {
        for (int j = sub + LPR; j < p.k; j += LPR) {
          int id2;
          float gw2;
          choice(r, j, id2, gw2);
          if (id2 >= 0) add[id2] = 0.0f;
        }
      }
      __syncwarp();
    }
  }
}

}  // namespace fg
