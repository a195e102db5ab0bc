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

#include "sm100_ptx.cuh"

namespace fg {

constexpr int kRouteThreads = 256;
constexpr int kRouteWarps = kRouteThreads / 32;
constexpr int kRouteMaxK = 32;
constexpr float kLog2e = 1.4426950408889634f;

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// Order-preserving key of a logit: larger logit, larger key; 0 for -inf and NaN (never chosen), and
// -0 and +0 alike.
__device__ __forceinline__ uint32_t logit_key(float v) {
  if (!(v > -INFINITY)) return 0u;
  const uint32_t u = __float_as_uint(v + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_logit(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? (key & 0x7FFFFFFFu) : ~key);
}

// e^(x - high), high the row's largest logit.  The difference is formed first: with the type's lowest
// value in every place of a row, a product with log2(e) before it would overflow.
__device__ __forceinline__ float softmax_exp(float x, float high) { return exp2f((x - high) * kLog2e); }

// Reductions over the LPR lanes that hold one row (LPR a power of two).
template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
template <int LPR>
__device__ __forceinline__ float row_max(float v) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
template <int LPR>
__device__ __forceinline__ uint32_t row_max_u32(uint32_t v) {
  if constexpr (LPR == 32) {
    return __reduce_max_sync(0xffffffffu, v);
  } else {
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
  }
}
template <int LPR>
__device__ __forceinline__ int row_min_s32(int v) {
  if constexpr (LPR == 32) {
    return __reduce_min_sync(0xffffffffu, v);
  } else {
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) v = min(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
  }
}

// Value i of lane `sub` of a row is column (i / V * LPR + sub) * V + i % V: V consecutive columns
// per load, the lanes side by side.
template <int LPR, int V>
__device__ __forceinline__ int route_col(int i, int sub) {
  return (i / V * LPR + sub) * V + i % V;
}

// One row's values of this lane; columns at or past E read as -inf.  V > 1: E % V == 0 and the rows
// 16-byte aligned (V * sizeof(T) == 16).
template <typename T, int LPR, int NPL, int V>
__device__ __forceinline__ void load_logits(const T* row, int E, int sub, float (&x)[NPL]) {
#pragma unroll
  for (int i = 0; i < NPL; i += V) {
    const int c = route_col<LPR, V>(i, sub);
    if constexpr (V == 1) {
      x[i] = c < E ? to_f32(row[c]) : -INFINITY;
    } else {
      if (c < E) {
        const uint4 raw = *reinterpret_cast<const uint4*>(row + c);
        const T* t = reinterpret_cast<const T*>(&raw);
#pragma unroll
        for (int v = 0; v < V; ++v) x[i + v] = to_f32(t[v]);
      } else {
#pragma unroll
        for (int v = 0; v < V; ++v) x[i + v] = -INFINITY;
      }
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

// Forward, one CTA per (chunk of rows, sequence).  LPR lanes hold a row, NPL values each, so a warp
// works on 32 / LPR rows at once.
template <typename T, int LPR, int NPL, int V>
__global__ void __launch_bounds__(kRouteThreads) moe_route_kernel(const RouteParams p) {
  constexpr int RPW = 32 / LPR;
  constexpr int EP = LPR * NPL;
  __shared__ int s_cnt[EP + 1];
  __shared__ float s_sum[kRouteWarps][EP];
  __shared__ float s_w[kRouteWarps][RPW][kRouteMaxK];
  __shared__ int s_id[kRouteWarps][RPW][kRouteMaxK];
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
  const int first = chunk * p.rows_per_chunk;
  const int last = min(p.T, first + p.rows_per_chunk);
  for (int r0 = first + warp * RPW; r0 < last; r0 += kRouteWarps * RPW) {
    const int r = r0 + rw;
    const size_t row = static_cast<size_t>(seq) * p.T + min(r, last - 1);
    const bool live = r < last && (!p.mask || p.mask[row]);
    float x[NPL];
    uint32_t key[NPL];
    load_logits<T, LPR, NPL, V>(static_cast<const T*>(p.logits) + row * p.E, p.E, sub, x);
    uint32_t best = 0;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      key[i] = live ? logit_key(x[i]) : 0u;
      best = max(best, key[i]);
    }
    best = row_max_u32<LPR>(best);
    const bool routed = best != 0;
    const float high = routed ? key_logit(best) : 0.0f;
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      x[i] = softmax_exp(x[i], high);
      sum += x[i];
    }
    sum = row_sum<LPR>(sum);
    const float inv = 1.0f / sum;
    if (routed) {
#pragma unroll
      for (int i = 0; i < NPL; ++i) acc[i] += x[i] * inv;
    }
    // the k largest keys, one at a time; among equal keys the lowest column
    float top = 0.0f;
    for (int j = 0; j < p.k; ++j) {
      int col = 0x7fffffff;
#pragma unroll
      for (int i = 0; i < NPL; ++i)
        if (key[i] == best) col = min(col, route_col<LPR, V>(i, sub));
      col = row_min_s32<LPR>(col);
      const float w = best ? softmax_exp(key_logit(best), high) : 0.0f;
      top += w;
      if (sub == j % LPR) {
        s_id[warp][rw][j] = best ? col : -1;
        s_w[warp][rw][j] = w;
      }
      uint32_t next = 0;
#pragma unroll
      for (int i = 0; i < NPL; ++i) {
        if (key[i] == best && route_col<LPR, V>(i, sub) == col) key[i] = 0;
        next = max(next, key[i]);
      }
      best = row_max_u32<LPR>(next);
    }
    __syncwarp();
    if (r < last) {
      const float scale = routed ? 1.0f / (p.renorm ? top : sum) : 0.0f;
      for (int j = sub; j < p.k; j += LPR) {
        const int id = s_id[warp][rw][j];
        p.ids[row * p.k + j] = id;
        p.weights[row * p.k + j] = id >= 0 ? s_w[warp][rw][j] * scale : 0.0f;
        if (id >= 0) atomicAdd(&s_cnt[id], 1);
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
    p.part_p[slot * p.E + e] = v;
    p.part_n[slot * (p.E + 1) + e] = s_cnt[e];
  }
  if (threadIdx.x == 0) p.part_n[slot * (p.E + 1) + p.E] = s_cnt[EP];
}

// Sums of the chunks of one sequence (in chunk order), then its counts, slopes and loss.
__global__ void __launch_bounds__(1024) moe_route_finish_kernel(const RouteParams p) {
  __shared__ float s_red[32];
  __shared__ int s_n[2];
  const int seq = blockIdx.x;
  if (threadIdx.x < 2) s_n[threadIdx.x] = 0;
  __syncthreads();
  pdl_wait_prior_grid();
  pdl_launch_dependents();
  const size_t slot = static_cast<size_t>(seq) * p.chunks;
  const int e = threadIdx.x;
  float sum = 0.0f;
  int n = 0;
  if (e < p.E) {
    for (int c = 0; c < p.chunks; ++c) {
      sum += p.part_p[(slot + c) * p.E + e];
      n += p.part_n[(slot + c) * (p.E + 1) + e];
    }
    p.counts[static_cast<size_t>(seq) * p.E + e] = n;
    if (n) atomicAdd(&s_n[0], n);
  }
  int rows = 0;
  for (int c = e; c < p.chunks; c += blockDim.x) rows += p.part_n[(slot + c) * (p.E + 1) + p.E];
  if (rows) atomicAdd(&s_n[1], rows);
  __syncthreads();
  const float total = static_cast<float>(max(s_n[0], 1)) * static_cast<float>(max(s_n[1], 1));
  const float slope = static_cast<float>(p.E) * static_cast<float>(n) / total;
  if (e < p.E) p.slope[static_cast<size_t>(seq) * p.E + e] = slope;
  float v = row_sum<32>(e < p.E ? slope * sum : 0.0f);
  if ((threadIdx.x & 31) == 0) s_red[threadIdx.x >> 5] = v;
  __syncthreads();
  if (threadIdx.x < 32) {
    v = row_sum<32>(threadIdx.x < blockDim.x / 32 ? s_red[threadIdx.x] : 0.0f);
    if (threadIdx.x == 0) p.loss[seq] = v;
  }
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

// Backward.  With h_e = grad_loss * slope_e (+ grad_weights_j at the chosen columns when the weights
// are not renormalised):  d l = p (h - sum p h).  Renormalised weights are the softmax w over the
// chosen logits: d l_j += w_j (g_j - sum w g) there.  Rows without a choice get zeros.
template <typename T, int LPR, int NPL, int V>
__global__ void __launch_bounds__(kRouteThreads) moe_route_backward_kernel(const RouteGradParams p) {
  constexpr int RPW = 32 / LPR;
  constexpr int EP = LPR * NPL;
  __shared__ float s_add[kRouteWarps][RPW][EP];  // what the chosen columns add; zero between rows
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane % LPR, rw = lane / LPR;
  const int seq = blockIdx.y;
  for (int i = threadIdx.x; i < kRouteWarps * RPW * EP; i += kRouteThreads) (&s_add[0][0][0])[i] = 0.0f;
  __syncthreads();
  pdl_wait_prior_grid();
  pdl_launch_dependents();
  float* add = s_add[warp][rw];
  float h0[NPL];
  const float g = p.grad_loss ? p.grad_loss[seq] : 0.0f;
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const int c = route_col<LPR, V>(i, sub);
    h0[i] = p.grad_loss && c < p.E ? g * p.slope[static_cast<size_t>(seq) * p.E + c] : 0.0f;
  }
  const int first = blockIdx.x * p.rows_per_chunk;
  const int last = min(p.T, first + p.rows_per_chunk);
  for (int r0 = first + warp * RPW; r0 < last; r0 += kRouteWarps * RPW) {
    const int r = r0 + rw;
    const size_t row = static_cast<size_t>(seq) * p.T + min(r, last - 1);
    const T* logits = static_cast<const T*>(p.logits) + row * p.E;
    const int* ids = p.ids + row * p.k;
    float x[NPL];
    load_logits<T, LPR, NPL, V>(logits, p.E, sub, x);
    bool any = false;
    for (int j = sub; j < p.k; j += LPR) any |= ids[j] >= 0 && ids[j] < p.E;
    const bool routed = row_max<LPR>(any ? 1.0f : 0.0f) > 0.0f;
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < NPL; ++i) m = fmaxf(m, x[i]);
    const float high = row_max<LPR>(m);
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      x[i] = softmax_exp(x[i], high);
      sum += x[i];
    }
    const float inv = 1.0f / row_sum<LPR>(sum);
    if (p.grad_weights) {
      const float* gw = p.grad_weights + row * p.k;
      float top = 0.0f, dot = 0.0f;
      if (p.renorm) {
        for (int j = sub; j < p.k; j += LPR) {
          const int id = ids[j];
          if (id < 0 || id >= p.E) continue;
          const float w = softmax_exp(to_f32(logits[id]), high);
          top += w;
          dot += w * gw[j];
        }
        top = 1.0f / row_sum<LPR>(top);
        dot = row_sum<LPR>(dot) * top;
      }
      for (int j = sub; j < p.k; j += LPR) {
        const int id = ids[j];
        if (id < 0 || id >= p.E) continue;
        atomicAdd(&add[id], p.renorm ? softmax_exp(to_f32(logits[id]), high) * top * (gw[j] - dot) : gw[j]);
      }
      __syncwarp();
    }
    float dot = 0.0f;
    float a[NPL];
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      a[i] = add[route_col<LPR, V>(i, sub)];
      x[i] *= inv;
      dot += x[i] * (p.renorm ? h0[i] : h0[i] + a[i]);
    }
    dot = row_sum<LPR>(dot);
    __syncwarp();
    if (p.grad_weights) {
      for (int j = sub; j < p.k; j += LPR) {
        const int id = ids[j];
        if (id >= 0 && id < p.E) add[id] = 0.0f;
      }
      __syncwarp();
    }
    if (r >= last) continue;
    T* out = static_cast<T*>(p.grad_logits) + row * p.E;
#pragma unroll
    for (int i = 0; i < NPL; i += V) {
      const int c = route_col<LPR, V>(i, sub);
      if (c >= p.E) continue;
      alignas(16) T t[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float d = p.renorm ? x[i + v] * (h0[i + v] - dot) + a[i + v]
                                 : x[i + v] * (h0[i + v] + a[i + v] - dot);
        t[v] = from_f32<T>(routed ? d : 0.0f);
      }
      if constexpr (V == 1)
        out[c] = t[0];
      else
        *reinterpret_cast<uint4*>(out + c) = *reinterpret_cast<const uint4*>(t);
    }
  }
}

}  // namespace fg
