// lora_kernels.cuh -- low-rank adapters of many requests at once beside a shared projection:
//   out[m] = C[m] + scaling[a] * B_a (A_a x[m]),  a = adapter of row m (none: out[m] = C[m]),
// x bf16 [M, K], A bf16 [L, R, K], B bf16 [L, N, R], C and out bf16 [M, N].
#pragma once

#include <cuda_bf16.h>
#include <cstdint>

#include "cluster_ptx.cuh"
#include "sm100_ptx.cuh"

namespace fg {

constexpr int kLoraThreads = 256;
constexpr int kLoraWarps = kLoraThreads / 32;
constexpr int kLoraCluster = 8;
constexpr int kLoraMaxRank = 128;

struct LoraParams {
  const __nv_bfloat16* C;
  const __nv_bfloat16* x;
  const __nv_bfloat16* a;
  const __nv_bfloat16* b;
  const int* adapters;   // [M]
  const float* scaling;  // [L] or nullptr (all 1)
  __nv_bfloat16* out;
  int M, N, K, R, L;
};

// D += A B, one 16 x 8 x 16 bf16 product of a warp with fp32 accumulators.
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// (hi, lo) bf16 pairs of two fp32 values: hi + lo is within 2^-16 of the value, relative.  An
// infinity or a NaN stays in hi alone (inf - inf would make a NaN of lo).
__device__ __forceinline__ float bf16_rest(float v, float hi) { return fabsf(hi) < INFINITY ? v - hi : 0.0f; }
__device__ __forceinline__ void split_bf16x2(float v0, float v1, uint32_t& hi, uint32_t& lo) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(v0, v1);
  const __nv_bfloat162 l = __floats2bfloat162_rn(bf16_rest(v0, __low2float(h)), bf16_rest(v1, __high2float(h)));
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = *reinterpret_cast<const uint32_t*>(&l);
}

// Up to 16 rows of one adapter per cluster of eight CTAs, for few rows.  Cluster m belongs to row m
// and works if the row is the first of a group of 16 among the rows of its adapter.  A rank of the
// cluster takes an eighth of K for h = A x (its warps strided over 32-wide blocks), the parts are
// summed through distributed shared memory in rank order, and each rank then takes an eighth of N.
// NT: eights of the rank held (R <= 8 NT).
template <int NT>
__global__ void __launch_bounds__(kLoraThreads) lora_rows_kernel(const LoraParams p) {
  constexpr int RP = NT * 8;
  extern __shared__ float s_dyn[];
  float* s_part = s_dyn;                          // [warps][16][RP], then the sum over the warps in [0]
  float* s_h = s_dyn + kLoraWarps * 16 * RP;      // [16][RP]
  __shared__ int s_rows[16];
  __shared__ int s_cnt[kLoraWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, q = lane & 3;
  const int rank = static_cast<int>(cluster_ctarank());
  const int m0 = blockIdx.x / kLoraCluster;
  pdl_wait_prior_grid();
  pdl_launch_dependents();
  int ad = p.adapters[m0];
  if (ad < 0 || ad >= p.L) ad = -1;
  if (ad < 0 && p.out == p.C) return;
  // place of row m0 among the rows of its adapter, then the rows of its group
  int before = 0;
  for (int m = threadIdx.x; m < m0; m += kLoraThreads) {
    const int v = p.adapters[m];
    before += ad < 0 ? (v < 0 || v >= p.L) : v == ad;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
  if (lane == 0) s_cnt[warp] = before;
  if (threadIdx.x < 16) s_rows[threadIdx.x] = -1;
  __syncthreads();
  before = 0;
#pragma unroll
  for (int w = 0; w < kLoraWarps; ++w) before += s_cnt[w];
  if (before % 16 != 0) return;
  int found = 0;
  for (int base = m0; base < p.M && found < 16; base += kLoraThreads) {
    __syncthreads();
    const int m = base + threadIdx.x;
    const int v = m < p.M ? p.adapters[m] : 0;
    const bool mine = m < p.M && (ad < 0 ? (v < 0 || v >= p.L) : v == ad);
    const uint32_t vote = __ballot_sync(0xffffffffu, mine);
    if (lane == 0) s_cnt[warp] = __popc(vote);
    __syncthreads();
    int at = found + __popc(vote & ((1u << lane) - 1));
#pragma unroll
    for (int w = 0; w < kLoraWarps; ++w) {
      if (w < warp) at += s_cnt[w];
      found += s_cnt[w];
    }
    if (mine && at < 16) s_rows[at] = m;
  }
  __syncthreads();
  const int row0 = s_rows[g], row1 = s_rows[g + 8];
  const int groups = (p.N + 31) / 32;
  const int g0 = static_cast<int>(static_cast<long long>(groups) * rank / kLoraCluster);
  const int g1 = static_cast<int>(static_cast<long long>(groups) * (rank + 1) / kLoraCluster);

  if (ad < 0) {  // no adapter: the rows are copied
    for (int gr = g0 + warp; gr < g1; gr += kLoraWarps) {
      const int col = gr * 32 + q * 8;
      if (col >= p.N) continue;
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const int row = s ? row1 : row0;
        if (row < 0) continue;
        const size_t at = static_cast<size_t>(row) * p.N + col;
        *reinterpret_cast<uint4*>(p.out + at) = *reinterpret_cast<const uint4*>(p.C + at);
      }
    }
    return;
  }

  // h = A x over this rank's part of K.  The lane's eight consecutive values of a 32-wide block feed
  // two 16-wide products (the order of k inside a product is free as long as both operands agree).
  float acc[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[n][i] = 0.0f;
  const int kblocks = (p.K + 31) / 32;
  const int k0 = static_cast<int>(static_cast<long long>(kblocks) * rank / kLoraCluster);
  const int k1 = static_cast<int>(static_cast<long long>(kblocks) * (rank + 1) / kLoraCluster);
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  const __nv_bfloat16* wa = p.a + static_cast<size_t>(ad) * p.R * p.K;
  for (int kb = k0 + warp; kb < k1; kb += kLoraWarps) {
    const int k = kb * 32 + q * 8;
    const bool in = k < p.K;
    const uint4 x0 = in && row0 >= 0 ? __ldg(reinterpret_cast<const uint4*>(p.x + static_cast<size_t>(row0) * p.K + k)) : zero;
    const uint4 x1 = in && row1 >= 0 ? __ldg(reinterpret_cast<const uint4*>(p.x + static_cast<size_t>(row1) * p.K + k)) : zero;
    uint4 w[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int r = n * 8 + g;
      w[n] = in && r < p.R ? __ldg(reinterpret_cast<const uint4*>(wa + static_cast<size_t>(r) * p.K + k)) : zero;
    }
    const uint32_t f0[4] = {x0.x, x1.x, x0.y, x1.y}, f1[4] = {x0.z, x1.z, x0.w, x1.w};
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      mma_16816(acc[n], f0, w[n].x, w[n].y);
      mma_16816(acc[n], f1, w[n].z, w[n].w);
    }
  }
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    float* part = s_part + warp * 16 * RP + n * 8 + q * 2;
    part[g * RP] = acc[n][0];
    part[g * RP + 1] = acc[n][1];
    part[(g + 8) * RP] = acc[n][2];
    part[(g + 8) * RP + 1] = acc[n][3];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 16 * RP; i += kLoraThreads) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kLoraWarps; ++w) v += s_part[w * 16 * RP + i];
    s_part[i] = v;
  }
  cluster_sync_all();
  const float scale = p.scaling ? p.scaling[ad] : 1.0f;
  const uint32_t part = smem_addr(s_part);
  for (int i = threadIdx.x; i < 16 * RP; i += kLoraThreads) {
    float v = 0.0f;
#pragma unroll
    for (int c = 0; c < kLoraCluster; ++c) v += ld_dsmem_f32(mapa_shared(part + i * 4, c));
    s_h[i] = v * scale;
  }
  cluster_sync_all();  // every rank has read the parts; s_h is complete

  // delta = h B^T.  Both bf16 halves of h go through the tensor cores, so h keeps 16 bits.  Column
  // 8 q + 2 i + b of a 32-wide group is column 2 q + b of product i: a lane owns eight consecutive
  // columns of two rows.
  constexpr int NS = (NT + 1) / 2;  // 16-wide steps over the rank
  uint32_t hi[NS][4], lo[NS][4];
#pragma unroll
  for (int s = 0; s < NS; ++s) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = s * 16 + q * 4 + (i >> 1) * 2, row = g + (i & 1) * 8;
      const bool in = r < RP;
      split_bf16x2(in ? s_h[row * RP + r] : 0.0f, in ? s_h[row * RP + r + 1] : 0.0f, hi[s][i], lo[s][i]);
    }
  }
  const __nv_bfloat16* wb = p.b + static_cast<size_t>(ad) * p.N * p.R;
  for (int gr = g0 + warp; gr < g1; gr += kLoraWarps) {
    float d[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int c = 0; c < 4; ++c) d[i][c] = 0.0f;
      const int n = gr * 32 + (g >> 1) * 8 + 2 * i + (g & 1);
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        const int r = s * 16 + q * 4;
        const uint2 w = n < p.N && r < p.R ? __ldg(reinterpret_cast<const uint2*>(wb + static_cast<size_t>(n) * p.R + r))
                                           : make_uint2(0u, 0u);
        mma_16816(d[i], hi[s], w.x, w.y);
        mma_16816(d[i], lo[s], w.x, w.y);
      }
    }
    const int col = gr * 32 + q * 8;
    if (col >= p.N) continue;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int row = s ? row1 : row0;
      if (row < 0) continue;
      const size_t at = static_cast<size_t>(row) * p.N + col;
      const uint4 raw = *reinterpret_cast<const uint4*>(p.C + at);
      const uint32_t c[4] = {raw.x, raw.y, raw.z, raw.w};
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float v0 = __uint_as_float(c[i] << 16) + d[i][2 * s];
        const float v1 = __uint_as_float(c[i] & 0xFFFF0000u) + d[i][2 * s + 1];
        const __nv_bfloat162 h = __floats2bfloat162_rn(v0, v1);
        o[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
      *reinterpret_cast<uint4*>(p.out + at) = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

}  // namespace fg
