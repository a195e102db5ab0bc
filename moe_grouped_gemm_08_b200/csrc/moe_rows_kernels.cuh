// moe_rows_kernels.cuh -- the rows' way to the experts and back: the experts' row layout, the cast
// of each token's row into it, the weighted sum of the experts' output rows, and its gradients.
//
// A pair is (token t, choice j), with the expert ids[t][j] or none (any value outside [0, E)).  Its
// row in the layout is rows[t][j], -1 for a pair without one.
#pragma once

#include <cuda_bf16.h>
#include <cstdint>

#include "fp8_cast_kernels.cuh"
#include "sm100_ptx.cuh"

namespace fg {

constexpr int kLayoutThreads = 256;
constexpr int kLayoutWarps = kLayoutThreads / 32;
constexpr int kLayoutItems = 8;                               // pairs per thread
constexpr int kLayoutChunk = kLayoutThreads * kLayoutItems;   // pairs per CTA
constexpr int kLayoutMaxExperts = 1024;
constexpr int kRowsMaxK = 32;

struct LayoutParams {
  const int* ids;  // [pairs]
  int* rows;       // [pairs]
  int* group;      // contiguous: m_indices [M]; masked: masked_m [E]
  int* hist;       // [chunks][E], unused with one chunk
  long long pairs;
  int E, chunks, M, mmax, align;  // mmax > 0: masked layout
};

// Counts per expert of one chunk of pairs.
__global__ void __launch_bounds__(kLayoutThreads) moe_layout_count_kernel(const LayoutParams p) {
  __shared__ int s_cnt[kLayoutMaxExperts];
  for (int e = threadIdx.x; e < p.E; e += kLayoutThreads) s_cnt[e] = 0;
  __syncthreads();
  pdl_wait_prior_grid();
  pdl_launch_dependents();
  const long long base = static_cast<long long>(blockIdx.x) * kLayoutChunk;
#pragma unroll
  for (int i = 0; i < kLayoutItems; ++i) {
    const long long at = base + i * kLayoutThreads + threadIdx.x;
    const int id = at < p.pairs ? p.ids[at] : -1;
    if (id >= 0 && id < p.E) atomicAdd(&s_cnt[id], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += kLayoutThreads)
    p.hist[static_cast<size_t>(blockIdx.x) * p.E + e] = s_cnt[e];
}

// The stable counting sort of a chunk: a pair's row is its expert's first row, plus the expert's
// pairs in earlier chunks, in earlier warps of the chunk, and earlier in its warp.
__global__ void __launch_bounds__(kLayoutThreads) moe_layout_kernel(const LayoutParams p) {
  __shared__ uint16_t s_warp[kLayoutWarps][kLayoutMaxExperts];  // counts, then prefixes over the warps
  __shared__ int s_start[kLayoutMaxExperts];  // the expert's first row
  __shared__ int s_count[kLayoutMaxExperts];  // its pairs
  __shared__ int s_before[kLayoutMaxExperts];  // its pairs in earlier chunks
  __shared__ int s_scan[kLayoutWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < kLayoutWarps * kLayoutMaxExperts; i += kLayoutThreads) (&s_warp[0][0])[i] = 0;
  __syncthreads();
  pdl_wait_prior_grid();
  pdl_launch_dependents();
  const long long base = static_cast<long long>(blockIdx.x) * kLayoutChunk + warp * 32 * kLayoutItems;
  int id[kLayoutItems], rank[kLayoutItems];
#pragma unroll
  for (int i = 0; i < kLayoutItems; ++i) {
    const long long at = base + i * 32 + lane;
    id[i] = at < p.pairs ? p.ids[at] : -1;
    if (id[i] >= p.E) id[i] = -1;
  }
#pragma unroll
  for (int i = 0; i < kLayoutItems; ++i) {
    const int e = id[i] < 0 ? -1 : id[i];
    const uint32_t same = __match_any_sync(0xffffffffu, e);
    const int before = e >= 0 ? s_warp[warp][e] : 0;
    rank[i] = before + __popc(same & ((1u << lane) - 1));
    __syncwarp();
    if (e >= 0 && lane == __ffs(same) - 1) s_warp[warp][e] = static_cast<uint16_t>(before + __popc(same));
    __syncwarp();
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += kLayoutThreads) {
    int run = 0;
#pragma unroll
    for (int w = 0; w < kLayoutWarps; ++w) {
      const int c = s_warp[w][e];
      s_warp[w][e] = static_cast<uint16_t>(run);
      run += c;
    }
    int before = 0, count = run;
    if (p.chunks > 1) {
      count = 0;
      for (int c = 0; c < p.chunks; ++c) {
        const int v = p.hist[static_cast<size_t>(c) * p.E + e];
        if (c < static_cast<int>(blockIdx.x)) before += v;
        count += v;
      }
    }
    s_before[e] = before;
    s_count[e] = count;
  }
  __syncthreads();
  // first rows: the experts' blocks one after the other, each padded to the alignment
  if (p.mmax > 0) {
    for (int e = threadIdx.x; e < p.E; e += kLayoutThreads) s_start[e] = e * p.mmax;
  } else {
    constexpr int PER = kLayoutMaxExperts / kLayoutThreads;
    int pad[PER], sum = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = threadIdx.x * PER + i;
      pad[i] = e < p.E ? (s_count[e] + p.align - 1) / p.align * p.align : 0;
      sum += pad[i];
    }
    int run = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += v;
    }
    if (lane == 31) s_scan[warp] = run;
    __syncthreads();
    run -= sum;
    for (int w = 0; w < warp; ++w) run += s_scan[w];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = threadIdx.x * PER + i;
      if (e < p.E) s_start[e] = run;
      run += pad[i];
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kLayoutItems; ++i) {
    const long long at = base + i * 32 + lane;
    if (at >= p.pairs) continue;
    const int e = id[i];
    int row = -1;
    if (e >= 0) {
      const int place = s_before[e] + s_warp[warp][e] + rank[i];
      if (p.mmax <= 0 || place < p.mmax) row = s_start[e] + place;
    }
    p.rows[at] = row;
  }
  if (p.mmax > 0) {
    if (blockIdx.x == 0)
      for (int e = threadIdx.x; e < p.E; e += kLayoutThreads) p.group[e] = min(s_count[e], p.mmax);
    return;
  }
  // m_indices: the last expert whose block starts at or before the row, if the row holds one of its
  // pairs (experts without pairs share their start with the next one and are passed over)
  for (int r = blockIdx.x * kLayoutThreads + threadIdx.x; r < p.M; r += gridDim.x * kLayoutThreads) {
    int lo = 0, hi = p.E;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s_start[mid] <= r) lo = mid; else hi = mid;
    }
    p.group[r] = r - s_start[lo] < s_count[lo] ? lo : -1;
  }
}

struct DispatchParams {
  const __nv_bfloat16* x;  // [T][K]
  const int* rows;         // [T][k]
  uint8_t* A;              // [M][K] or [G][mmax][K]
  float* sfa;              // [KB][ld] or [G][KB][ld]
  long long T;
  int k, K, M, mmax, ld;   // M: all rows of the layout; mmax: rows of a group (contiguous: M)
};

// One warp per token and 1024 columns: the row is read and cast once (as fp8_cast_rows_kernel
// does), then stored at each of its rows.
template <int FMT>
__global__ void __launch_bounds__(256) moe_dispatch_kernel(const DispatchParams p, int chunks) {
  const int lane = threadIdx.x & 31;
  const long long nwarps = (static_cast<long long>(gridDim.x) * blockDim.x) >> 5;
  const int KB = (p.K + 127) / 128;
  pdl_wait_prior_grid();
  pdl_launch_dependents();
  for (long long w = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5; w < p.T * chunks;
       w += nwarps) {
    const long long t = w / chunks;
    const int c = static_cast<int>(w - t * chunks);
    int mine = lane < p.k ? p.rows[t * p.k + lane] : -1;
    if (mine >= p.M) mine = -1;
    if (__ballot_sync(0xffffffffu, mine >= 0) == 0) continue;
    const __nv_bfloat16* xr = p.x + t * p.K;
    uint4 raw[kCastSpans];
#pragma unroll
    for (int j = 0; j < kCastSpans; ++j) {
      const int col = (c * kCastSpans + j) * 256 + lane * 8;
      raw[j] = col < p.K ? __ldg(reinterpret_cast<const uint4*>(xr + col)) : make_uint4(0u, 0u, 0u, 0u);
    }
    uint2 code[kCastSpans];
    float scale[kCastSpans];
#pragma unroll
    for (int j = 0; j < kCastSpans; ++j) {
      float f[8];
      unpack_bf16x8(raw[j], f);
      float amax = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(f[i]));
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      scale[j] = cast_scale<FMT>(amax);
      code[j] = encode_fp8x8<FMT>(f, scale[j]);
    }
    for (int q = 0; q < p.k; ++q) {
      const int row = __shfl_sync(0xffffffffu, mine, q);
      if (row < 0) continue;
      const int g = row / p.mmax, m = row - g * p.mmax;
#pragma unroll
      for (int j = 0; j < kCastSpans; ++j) {
        const int col = (c * kCastSpans + j) * 256 + lane * 8;
        if (col >= p.K) continue;
        *reinterpret_cast<uint2*>(p.A + static_cast<size_t>(row) * p.K + col) = code[j];
        if ((lane & 15) == 0) p.sfa[(static_cast<size_t>(g) * KB + col / 128) * p.ld + m] = scale[j];
      }
    }
  }
}

struct CombineParams {
  const __nv_bfloat16* C;  // [M][N]
  const int* rows;         // [T][k]
  const float* weights;    // [T][k] or nullptr (all 1)
  __nv_bfloat16* out;      // [T][N]
  long long T;
  int k, N, M;
};

__device__ __forceinline__ uint4 pack_bf16x8(const float (&f)[8]) {
  __nv_bfloat162 h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
  return *reinterpret_cast<const uint4*>(h);
}

// out[t] = sum_j weights[t][j] C[rows[t][j]] in fp32, rounded once.  One warp per token and 256
// columns, 8 per lane.
__global__ void __launch_bounds__(256) moe_combine_kernel(const CombineParams p, int chunks) {
  const int lane = threadIdx.x & 31;
  const long long nwarps = (static_cast<long long>(gridDim.x) * blockDim.x) >> 5;
  pdl_wait_prior_grid();
  pdl_launch_dependents();
  for (long long w = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5; w < p.T * chunks;
       w += nwarps) {
    const long long t = w / chunks;
    const int col = static_cast<int>(w - t * chunks) * 256 + lane * 8;
    int mine = lane < p.k ? p.rows[t * p.k + lane] : -1;
    if (mine >= p.M) mine = -1;
    const float mw = mine >= 0 ? (p.weights ? p.weights[t * p.k + lane] : 1.0f) : 0.0f;
    float acc[8] = {};
    for (int q = 0; q < p.k; ++q) {
      const int row = __shfl_sync(0xffffffffu, mine, q);
      const float wq = __shfl_sync(0xffffffffu, mw, q);
      if (row < 0 || col >= p.N) continue;
      float f[8];
      unpack_bf16x8(__ldg(reinterpret_cast<const uint4*>(p.C + static_cast<size_t>(row) * p.N + col)), f);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = fmaf(wq, f[i], acc[i]);
    }
    if (col < p.N) *reinterpret_cast<uint4*>(p.out + t * p.N + col) = pack_bf16x8(acc);
  }
}

struct CombineGradParams {
  const __nv_bfloat16* grad_out;  // [T][N]
  const __nv_bfloat16* C;         // [M][N]
  const int* rows;                // [T][k]
  const float* weights;           // [T][k]
  __nv_bfloat16* grad_C;          // [M][N]
  float* grad_weights;            // [T][k]
  long long T;
  int k, N, M;
};

// grad_C[rows[t][j]] = weights[t][j] grad_out[t];  grad_weights[t][j] = <grad_out[t], C[rows[t][j]]>.
// One CTA per token; eight choices at a time, their dot products in registers.
__global__ void __launch_bounds__(256) moe_combine_backward_kernel(const CombineGradParams p) {
  __shared__ float s_dot[8][8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait_prior_grid();
  pdl_launch_dependents();
  for (long long t = blockIdx.x; t < p.T; t += gridDim.x) {
    for (int j0 = 0; j0 < p.k; j0 += 8) {
      int row[8];
      float w[8], dot[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        row[j] = j0 + j < p.k ? p.rows[t * p.k + j0 + j] : -1;
        if (row[j] >= p.M) row[j] = -1;
        w[j] = row[j] >= 0 ? p.weights[t * p.k + j0 + j] : 0.0f;
        dot[j] = 0.0f;
      }
      for (int col = threadIdx.x * 8; col < p.N; col += 256 * 8) {
        float g[8];
        unpack_bf16x8(__ldg(reinterpret_cast<const uint4*>(p.grad_out + t * p.N + col)), g);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (row[j] < 0) continue;
          const size_t at = static_cast<size_t>(row[j]) * p.N + col;
          float f[8], o[8];
          unpack_bf16x8(__ldg(reinterpret_cast<const uint4*>(p.C + at)), f);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            dot[j] = fmaf(g[i], f[i], dot[j]);
            o[i] = w[j] * g[i];
          }
          *reinterpret_cast<uint4*>(p.grad_C + at) = pack_bf16x8(o);
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], o);
        if (lane == 0) s_dot[warp][j] = dot[j];
      }
      __syncthreads();
      if (threadIdx.x < 8 && j0 + static_cast<int>(threadIdx.x) < p.k) {
        float v = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) v += s_dot[i][threadIdx.x];
        p.grad_weights[t * p.k + j0 + threadIdx.x] = v;
      }
      __syncthreads();
    }
  }
}

}  // namespace fg
