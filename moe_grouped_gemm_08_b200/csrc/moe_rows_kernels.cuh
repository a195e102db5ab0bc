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

constexpr int kLayoutMaxExperts = 1024;
constexpr int kRowsMaxK = 32;

struct LayoutParams {
  const int* ids;  // [pairs]
  int* rows;       // [pairs]
  int* group;      // contiguous: m_indices [M]; masked: masked_m [E]
  int* hist;       // [chunks][E], unused with one chunk
  long long pairs;
  int E, chunks, M, mmax, align;  // mmax > 0: masked layout
  int* inverse;  // [M], the pair of each occupied row; nullptr: not wanted (then rows is)
  int rest;      // 1: ids outside [0, E - 1) are expert E - 1; 0: they have no row
  int* tiles;    // with rest: blocks of `align` rows of the experts below E - 1, and of all
};

__device__ __forceinline__ int layout_id(const LayoutParams& p, long long at) {
  if (at >= p.pairs) return -1;
  const int id = p.ids[at], none = p.rest ? p.E - 1 : -1;
  return id >= 0 && id < p.E - p.rest ? id : none;
}

// Counts per expert of one chunk of pairs (THREADS * ITEMS, in their order).
template <int THREADS, int ITEMS>
__global__ void __launch_bounds__(THREADS) moe_layout_count_kernel(const LayoutParams p) {
  __shared__ int s_cnt[kLayoutMaxExperts];
  for (int e = threadIdx.x; e < p.E; e += THREADS) s_cnt[e] = 0;
  __syncthreads();
  pdl_wait_prior_grid();
  pdl_launch_dependents();
  const long long base = static_cast<long long>(blockIdx.x) * (THREADS * ITEMS);
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const long long at = base + i * THREADS + threadIdx.x;
    const int id = layout_id(p, at);
    if (id >= 0) atomicAdd(&s_cnt[id], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += THREADS)
    p.hist[static_cast<size_t>(blockIdx.x) * p.E + e] = s_cnt[e];
}

// 512 pairs of 8 experts take 2.8 us (latency: one launch), 32768 of 256 experts 8.3 us (two).
// More CTAs than chunks help to fill m_indices: with one chunk all of them count it, with several they
// read the counts; only the chunk's own CTA writes its rows.  The stable counting sort of a chunk: a pair's row is its expert's first row, plus the expert's
// pairs in earlier chunks, in earlier warps of the chunk, and earlier in its warp.
template <int THREADS, int ITEMS>
__global__ void __launch_bounds__(THREADS) moe_layout_kernel(const LayoutParams p) {
  constexpr int WARPS = THREADS / 32;
  extern __shared__ uint16_t s_warp_counts[];  // [WARPS][E]: counts, then prefixes over the warps
  __shared__ int s_start[kLayoutMaxExperts];   // the expert's first row
  __shared__ int s_count[kLayoutMaxExperts];   // its pairs
  __shared__ int s_before[kLayoutMaxExperts];  // its pairs in earlier chunks
  __shared__ int s_scan[WARPS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int e = threadIdx.x; e < p.E; e += THREADS) {
#pragma unroll
    for (int w = 0; w < WARPS; ++w) s_warp_counts[w * p.E + e] = 0;
    s_before[e] = 0;
    s_count[e] = 0;
  }
  __syncthreads();
  pdl_wait_prior_grid();
  pdl_launch_dependents();
  const int chunk = p.chunks > 1 ? blockIdx.x : 0;
  const long long base = static_cast<long long>(chunk) * (THREADS * ITEMS) + warp * 32 * ITEMS;
  int id[ITEMS], rank[ITEMS];
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    id[i] = layout_id(p, base + i * 32 + lane);
  }
  if (p.chunks > 1) {  // all threads over (chunk, expert), as many chunks side by side as there is room
    const int cols = p.E < 32 ? 32 : p.E < THREADS ? (p.E + 31) / 32 * 32 : THREADS;
    const int parts = THREADS / cols;
    const int part = threadIdx.x / cols;
    for (int e = threadIdx.x % cols; e < p.E && part < parts; e += cols) {
      int before = 0, count = 0;
#pragma unroll 8
      for (int c = part; c < p.chunks; c += parts) {
        const int v = p.hist[static_cast<size_t>(c) * p.E + e];
        before += c < static_cast<int>(blockIdx.x) ? v : 0;
        count += v;
      }
      atomicAdd(&s_before[e], before);
      atomicAdd(&s_count[e], count);
    }
  }
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int e = id[i];
    const uint32_t same = __match_any_sync(0xffffffffu, e);
    const int before = e >= 0 ? s_warp_counts[warp * p.E + e] : 0;
    rank[i] = before + __popc(same & ((1u << lane) - 1));
    __syncwarp();
    if (e >= 0 && lane == __ffs(same) - 1) s_warp_counts[warp * p.E + e] = static_cast<uint16_t>(before + __popc(same));
    __syncwarp();
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += THREADS) {
    int run = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      const int c = s_warp_counts[w * p.E + e];
      s_warp_counts[w * p.E + e] = static_cast<uint16_t>(run);
      run += c;
    }
    if (p.chunks <= 1) s_count[e] = run;
  }
  __syncthreads();
  // first rows: the experts' blocks one after the other, each padded to the alignment
  if (p.mmax > 0) {
    for (int e = threadIdx.x; e < p.E; e += THREADS) s_start[e] = e * p.mmax;
  } else {
    constexpr int PER = kLayoutMaxExperts / THREADS;
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
  for (int i = 0; i < ITEMS; ++i) {
    const long long at = base + i * 32 + lane;
    if (at >= p.pairs || (p.chunks <= 1 && blockIdx.x > 0)) continue;
    const int e = id[i];
    int row = -1;
    if (e >= 0) {
      const int place = s_before[e] + s_warp_counts[warp * p.E + e] + rank[i];
      if (p.mmax <= 0 || place < p.mmax) row = s_start[e] + place;
    }
    if (p.inverse)
      p.inverse[row] = static_cast<int>(at);  // with `rest` every pair has a row
    else
      p.rows[at] = row;
  }
  if (p.mmax > 0) {
    if (blockIdx.x == 0)
      for (int e = threadIdx.x; e < p.E; e += THREADS) p.group[e] = min(s_count[e], p.mmax);
    return;
  }
  if (p.rest && blockIdx.x == 0 && threadIdx.x < 2) {
    const int total = s_start[p.E - 1] + (s_count[p.E - 1] + p.align - 1) / p.align * p.align;
    p.tiles[threadIdx.x] = (threadIdx.x ? total : s_start[p.E - 1]) / p.align;
  }
  // m_indices, four rows at a time (a block is a multiple of four): the last expert whose block starts at or
  // before the row, if the row holds one of its pairs (experts without pairs share their start with the
  // next one and are passed over).  r in 64 bits: M may be the largest int.
  for (long long r = (blockIdx.x * THREADS + threadIdx.x) * 4; r < p.M; r += gridDim.x * THREADS * 4) {
    int lo = 0, hi = p.E;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s_start[mid] <= r) lo = mid; else hi = mid;
    }
    const int left = static_cast<int>(s_start[lo] + s_count[lo] - r);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (r + i < p.M) p.group[r + i] = i < left ? lo : -1;
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

// The FP8 codes of 16 values of one block.  The definition is the format's rounding of RN(x / scale).
// Inside the range below, q = RN(x r), r = RN(1 / scale), corrected once by its remainder (Markstein, "Computation
// of elementary functions on the IBM RISC System/6000", 1990) is that quotient: for x of 8 significant
// bits and scale = RN(amax / 448) with amax of 8 bits it was checked for all 128 x 128 mantissas, and
// scaling both by powers of two changes nothing.  (Values so small that their remainder underflows
// are 0 in either format.)  The signs keep -0 as it is.
template <int FMT>
__device__ __forceinline__ uint4 encode_fp8x16(const float (&f)[16], float scale) {
  constexpr __nv_fp8_interpretation_t kind = FMT == 0 ? __NV_E4M3 : __NV_E5M2;
  uint32_t h[8];
  if (scale >= 0x1p-80f) {
    const float r = __frcp_rn(scale);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float q[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        q[j] = f[2 * i + j] * r;
        q[j] = fmaf(-fmaf(q[j], scale, -f[2 * i + j]), r, q[j]);
      }
      h[i] = static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(q[0], q[1]), __NV_SATFINITE, kind));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      h[i] = static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(
          make_float2(__fdiv_rn(f[2 * i], scale), __fdiv_rn(f[2 * i + 1], scale)), __NV_SATFINITE, kind));
  }
  return make_uint4(h[0] | (h[1] << 16), h[2] | (h[3] << 16), h[4] | (h[5] << 16), h[6] | (h[7] << 16));
}

// One warp per token and kDispatchSpans * 512 columns, 16 per lane, so eight lanes hold a 128-wide block:
// the row is read and cast once, then stored at each of its rows.  Bound by HBM: 16384 rows of 7168 to two places
// each, 477 MB, in 78 us with the division above and 16 bytes a store (120 us with an IEEE division a value
// and 8).
constexpr int kDispatchSpans = 2;
template <int FMT>
__global__ void __launch_bounds__(256) moe_dispatch_kernel(const DispatchParams p, int chunks) {
  const int lane = threadIdx.x & 31;
  const long long nwarps = (static_cast<long long>(gridDim.x) * blockDim.x) >> 5;
  const int KB = (p.K - 1) / 128 + 1;  // K > 0, and K + 127 may not fit
  pdl_wait_prior_grid();
  pdl_launch_dependents();
  for (long long w = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5; w < p.T * chunks;
       w += nwarps) {
    const long long t = w / chunks;
    const int c = static_cast<int>(w - t * chunks);
    int mine = lane < p.k ? p.rows[t * p.k + lane] : -1;
    if (mine >= p.M) mine = -1;
    const __nv_bfloat16* xr = p.x + t * p.K;
    const int col0 = c * (kDispatchSpans * 512) + lane * 16;
    uint4 raw[kDispatchSpans][2];
#pragma unroll
    for (int j = 0; j < kDispatchSpans; ++j) {
      const int col = col0 + j * 512;
#pragma unroll
      for (int h = 0; h < 2; ++h)
        raw[j][h] = col < p.K ? __ldg(reinterpret_cast<const uint4*>(xr + col) + h) : make_uint4(0u, 0u, 0u, 0u);
    }
    uint32_t left = __ballot_sync(0xffffffffu, mine >= 0);
    if (left == 0) continue;
    uint4 code[kDispatchSpans];
    float scale[kDispatchSpans];
#pragma unroll
    for (int j = 0; j < kDispatchSpans; ++j) {
      float lo[8], hi[8], f[16];
      unpack_bf16x8(raw[j][0], lo);
      unpack_bf16x8(raw[j][1], hi);
      float amax = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        f[i] = lo[i];
        f[8 + i] = hi[i];
        amax = fmaxf(amax, fmaxf(fabsf(lo[i]), fabsf(hi[i])));
      }
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      scale[j] = cast_scale<FMT>(amax);
      code[j] = encode_fp8x16<FMT>(f, scale[j]);
    }
    for (; left; left &= left - 1) {
      const int row = __shfl_sync(0xffffffffu, mine, __ffs(left) - 1);
      const int g = row / p.mmax, m = row - g * p.mmax;
      uint8_t* dst = p.A + static_cast<size_t>(row) * p.K + col0;
      float* sdst = p.sfa + (static_cast<size_t>(g) * KB + col0 / 128) * p.ld + m;
#pragma unroll
      for (int j = 0; j < kDispatchSpans; ++j) {
        if (col0 + j * 512 >= p.K) continue;
        *reinterpret_cast<uint4*>(dst + j * 512) = code[j];
        if ((lane & 7) == 0) sdst[static_cast<size_t>(4 * j) * p.ld] = scale[j];
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

// out[t] = sum_j weights[t][j] C[rows[t][j]] in fp32, rounded once, in the order of j.  One warp per token and V
// vectors of 8 columns per lane, J choices at a time, J V = 8: all eight vectors are asked for before the first is
// used, and the next token's rows and weights are loaded meanwhile.  Bound by HBM: 705 MB in 105 us (2 choices of
// 7168 columns, J = 2; 124 us with one vector a lane and 64 warps an SM), 151 MB in 26 us (8 choices of
// 2048, J = 4; 29 us with J = 8).
template <int J>
__global__ void __launch_bounds__(256, 3) moe_combine_kernel(const CombineParams p, int chunks) {
  constexpr int V = 8 / J;
  const int lane = threadIdx.x & 31;
  const long long nwarps = (static_cast<long long>(gridDim.x) * blockDim.x) >> 5;
  const long long items = p.T * chunks;
  pdl_wait_prior_grid();
  pdl_launch_dependents();
  long long w = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  int row_next = -1;
  float w_next = 0.0f;
  auto fetch = [&](long long item) {
    const long long t = item / chunks;
    row_next = lane < p.k ? p.rows[t * p.k + lane] : -1;
    if (row_next >= p.M) row_next = -1;
    w_next = !p.weights ? 1.0f : lane < p.k ? p.weights[t * p.k + lane] : 0.0f;
  };
  if (w < items) fetch(w);
  for (; w < items; w += nwarps) {
    const long long t = w / chunks;
    const int col0 = static_cast<int>(w - t * chunks) * (V * 256) + lane * 8;
    const int mine = row_next;
    const float mw = w_next;
    if (w + nwarps < items) fetch(w + nwarps);
    float acc[V][8] = {};
    for (int q0 = 0; q0 < p.k; q0 += J) {
      uint4 raw[J][V];
#pragma unroll
      for (int q = 0; q < J; ++q) {
        const int row = q0 + q < p.k ? __shfl_sync(0xffffffffu, mine, q0 + q) : -1;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const int col = col0 + v * 256;
          raw[q][v] = row >= 0 && col < p.N
                          ? __ldg(reinterpret_cast<const uint4*>(p.C + static_cast<size_t>(row) * p.N + col))
                          : make_uint4(0u, 0u, 0u, 0u);
        }
      }
#pragma unroll
      for (int q = 0; q < J; ++q) {
        if (q0 + q >= p.k) break;
        const int row = __shfl_sync(0xffffffffu, mine, q0 + q);
        const float wq = __shfl_sync(0xffffffffu, mw, q0 + q);
        if (row < 0) continue;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          float f[8];
          unpack_bf16x8(raw[q][v], f);
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[v][i] = fmaf(wq, f[i], acc[v][i]);
        }
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (col0 + v * 256 < p.N) *reinterpret_cast<uint4*>(p.out + t * p.N + col0 + v * 256) = pack_bf16x8(acc[v]);
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

// Sums of eight values over a warp; lane 4 j gets the j-th.  Each step halves the values, not only the lanes.
__device__ __forceinline__ float warp_sum8(float (&v)[8], int lane) {
  float a[4], b[2];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool up = lane & 16;
    a[i] = (up ? v[i + 4] : v[i]) + __shfl_xor_sync(0xffffffffu, up ? v[i] : v[i + 4], 16);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const bool up = lane & 8;
    b[i] = (up ? a[i + 2] : a[i]) + __shfl_xor_sync(0xffffffffu, up ? a[i] : a[i + 2], 8);
  }
  const bool up = lane & 4;
  float c = (up ? b[1] : b[0]) + __shfl_xor_sync(0xffffffffu, up ? b[0] : b[1], 4);
  c += __shfl_xor_sync(0xffffffffu, c, 2);
  return c + __shfl_xor_sync(0xffffffffu, c, 1);
}

// grad_C[rows[t][j]] = weights[t][j] grad_out[t];  grad_weights[t][j] = <grad_out[t], C[rows[t][j]]>.
// One CTA per token and J choices, V vectors of 8 columns per thread and pass, J V = 8: all eight vectors of C
// are asked for before the first is used, and the next token's rows and weights are loaded meanwhile;
// dot products in registers.  Bound by HBM: 285 MB in 48 us (8 choices of 2048 columns), 1.17 GB in 192 us (2 of
// 7168).
constexpr int kCombineGradThreads = 256;
template <int J>
__global__ void __launch_bounds__(kCombineGradThreads, 3) moe_combine_backward_kernel(const CombineGradParams p) {
  constexpr int W = kCombineGradThreads / 32, V = 8 / J, SPAN = kCombineGradThreads * 8;
  __shared__ float s_dot[2][W][8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int buf = 0;
  pdl_wait_prior_grid();
  pdl_launch_dependents();
  const int groups = (p.k + J - 1) / J;
  const long long items = p.T * groups;  // a token and J of its choices
  int row_next = -1;
  float w_next = 0.0f;
  auto fetch = [&](long long item) {
    const long long t = groups == 1 ? item : item / groups;
    const int j = static_cast<int>(item - t * groups) * J + lane % J;
    row_next = j < p.k ? p.rows[t * p.k + j] : -1;
    if (row_next >= p.M) row_next = -1;
    w_next = j < p.k ? p.weights[t * p.k + j] : 0.0f;
  };
  if (blockIdx.x < items) fetch(blockIdx.x);
  for (long long item = blockIdx.x; item < items; item += gridDim.x) {
    const long long t = groups == 1 ? item : item / groups;
    const int j0 = static_cast<int>(item - t * groups) * J;
    const int mine = row_next;
    const float mw = w_next;
    if (item + gridDim.x < items) fetch(item + gridDim.x);
    float dot[8] = {};
    // unsigned: the step past the last columns may reach 2^31, at which V SPAN ends a pass exactly
    for (unsigned c0 = 0; c0 < static_cast<unsigned>(p.N); c0 += V * SPAN) {
      const int col0 = static_cast<int>(c0) + threadIdx.x * 8;
      const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
      uint4 graw[V], raw[V][J];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int col = col0 + v * SPAN;
        graw[v] = col < p.N ? __ldg(reinterpret_cast<const uint4*>(p.grad_out + t * p.N + col)) : zero;
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const int row = __shfl_sync(0xffffffffu, mine, j);
          raw[v][j] = row >= 0 && col < p.N
                          ? __ldg(reinterpret_cast<const uint4*>(p.C + static_cast<size_t>(row) * p.N + col)) : zero;
        }
      }
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int col = col0 + v * SPAN;
        float g[8];
        unpack_bf16x8(graw[v], g);
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const int row = __shfl_sync(0xffffffffu, mine, j);
          const float w = __shfl_sync(0xffffffffu, mw, j);
          if (row < 0) continue;  // its gradient stays 0, whatever grad_out holds
          float f[8], o[8];
          unpack_bf16x8(raw[v][j], f);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            dot[j] = fmaf(g[i], f[i], dot[j]);
            o[i] = w * g[i];
          }
          if (col < p.N)
            *reinterpret_cast<uint4*>(p.grad_C + static_cast<size_t>(row) * p.N + col) = pack_bf16x8(o);
        }
      }
    }
    const float sum8 = warp_sum8(dot, lane);
    if ((lane & 3) == 0) s_dot[buf][warp][lane >> 2] = sum8;
    __syncthreads();
    if (threadIdx.x < J && j0 + static_cast<int>(threadIdx.x) < p.k) {
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < W; ++i) sum += s_dot[buf][i][threadIdx.x];
      p.grad_weights[t * p.k + j0 + threadIdx.x] = sum;
    }
    buf ^= 1;  // the other buffer's readers are past the barrier above
  }
}

}  // namespace fg
