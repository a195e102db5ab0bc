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
  // many rows: places of the rows sorted by adapter, in tiles of 128
  const int* group;      // place -> adapter (L: none, -1: padding)
  const int* place_row;  // place -> row
  const int* tiles;      // tiles of adapters, tiles in all
  float* parts;          // [2 * CTAs + tiles][rank padded / 4][128][4]: two parts of h per CTA, whole h per tile
  int* status;
  int stall;  // test hook: the products' thread of lora_down_kernel (1) or lora_up_kernel (2) first waits for nothing
};

// D += A B, one 16 x 8 x 16 bf16 product of a warp with fp32 accumulators.
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two fp32 values as three pairs of bf16, cut off instead of rounded: each part takes eight bits of the significand,
// so that their sum is the value (but for bits below the normal numbers), and the first cannot overflow.
// An infinity or a NaN stays in the first part alone (inf - inf would make a NaN of the next).
constexpr int kLoraParts = 3;
__device__ __forceinline__ void split_bf16x2(float v0, float v1, uint32_t (&part)[kLoraParts]) {
#pragma unroll
  for (int i = 0; i < kLoraParts; ++i) {
    const uint32_t u0 = __float_as_uint(v0), u1 = __float_as_uint(v1);
    part[i] = __byte_perm(u0, u1, 0x7632);  // the upper halves
    const float h0 = __uint_as_float(u0 & 0xFFFF0000u), h1 = __uint_as_float(u1 & 0xFFFF0000u);
    v0 = fabsf(h0) < INFINITY ? v0 - h0 : 0.0f;
    v1 = fabsf(h1) < INFINITY ? v1 - h1 : 0.0f;
  }
}

// ---------------------------------------------------------------------------- few rows
// Up to 16 rows of one adapter per cluster of CL CTAs, one launch and no scratch.  Cluster m belongs to row m
// and works if the row is the first of a group of 16 among the rows of its adapter.  A rank of the
// cluster takes a CL-th of K for h = A x (its warps strided over 32-wide blocks), the parts are
// summed through distributed shared memory in rank order, and each rank then takes a CL-th of N.
// Bound by latency: the loads of a phase are all asked for before the first is used, and the first columns of
// B and C before h is ready.  K 7168, N 4096, rank 16: one row 4.6 us, 64 rows of 64 adapters 8.9, 128 rows 12.
// NT: eights of the rank held (R <= 8 NT).
template <int NT>
struct LoraRows {
  static constexpr int AHEAD = NT <= 2 ? 4 : NT <= 4 ? 2 : 1;  // blocks of K asked for at once
  static constexpr int CTAS = NT <= 4 ? 3 : NT <= 8 ? 2 : 1;   // per SM, for the registers
  static constexpr int LD = NT * 8 + (NT >= 4 ? 8 : 0);  // row of h in shared memory, floats: padded against bank conflicts
  static constexpr int SMEM = (kLoraWarps + 1) * 16 * LD * 4;
};
template <int NT, int CL>
__global__ void __launch_bounds__(kLoraThreads, LoraRows<NT>::CTAS) lora_rows_kernel(const LoraParams p) {
  constexpr int RP = NT * 8, AHEAD = LoraRows<NT>::AHEAD, LD = LoraRows<NT>::LD;
  extern __shared__ __align__(16) float s_dyn[];
  float* s_part = s_dyn;                      // [warps][16][LD], then the sum over the warps in [0]
  float* s_h = s_dyn + kLoraWarps * 16 * LD;  // [16][LD]
  __shared__ int s_rows[16];
  __shared__ int s_cnt[kLoraWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, q = lane & 3;
  const int rank = static_cast<int>(cluster_ctarank());
  const int m0 = blockIdx.x / CL;
  if (threadIdx.x < 16) s_rows[threadIdx.x] = -1;
  pdl_wait_prior_grid();
  pdl_launch_dependents();
  auto adapter = [&](int m) {
    const int v = p.adapters[m];
    return v >= 0 && v < p.L ? v : -1;
  };
  const int ad = adapter(m0);
  if (ad < 0 && p.out == p.C) return;
  // place of row m0 among the rows of its adapter, then the rows of its group
  int before = 0;
  for (int m = threadIdx.x; m < m0; m += kLoraThreads) before += adapter(m) == ad;
  before = __reduce_add_sync(0xffffffffu, before);
  if (lane == 0) s_cnt[warp] = before;
  __syncthreads();
  before = 0;
#pragma unroll
  for (int w = 0; w < kLoraWarps; ++w) before += s_cnt[w];
  if (before % 16 != 0) return;
  int found = 0;
  for (int base = m0; base < p.M && found < 16; base += kLoraThreads) {
    __syncthreads();
    const int m = base + threadIdx.x;
    const bool mine = m < p.M && adapter(m) == ad;
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
  const int groups = (p.N - 1) / 32 + 1;  // N > 0, and N + 31 may not fit; so for K
  const int g0 = static_cast<int>(static_cast<long long>(groups) * rank / CL);
  const int g1 = static_cast<int>(static_cast<long long>(groups) * (rank + 1) / CL);

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
  const int kblocks = (p.K - 1) / 32 + 1;
  const int k0 = static_cast<int>(static_cast<long long>(kblocks) * rank / CL);
  const int k1 = static_cast<int>(static_cast<long long>(kblocks) * (rank + 1) / CL);
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  const __nv_bfloat16* x0 = p.x + static_cast<size_t>(max(row0, 0)) * p.K + q * 8;
  const __nv_bfloat16* x1 = p.x + static_cast<size_t>(max(row1, 0)) * p.K + q * 8;
  const __nv_bfloat16* wa = p.a + (static_cast<size_t>(ad) * p.R + g) * p.K + q * 8;
  for (int kb = k0 + warp; kb < k1; kb += kLoraWarps * AHEAD) {
    uint4 xv[AHEAD][2], w[AHEAD][NT];
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      const int k = (kb + u * kLoraWarps) * 32;
      const bool in = kb + u * kLoraWarps < k1 && k + q * 8 < p.K;
      xv[u][0] = in && row0 >= 0 ? __ldg(reinterpret_cast<const uint4*>(x0 + k)) : zero;
      xv[u][1] = in && row1 >= 0 ? __ldg(reinterpret_cast<const uint4*>(x1 + k)) : zero;
#pragma unroll
      for (int n = 0; n < NT; ++n)
        w[u][n] = in && n * 8 + g < p.R ? __ldg(reinterpret_cast<const uint4*>(wa + static_cast<size_t>(n * 8) * p.K + k)) : zero;
    }
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      const uint32_t f0[4] = {xv[u][0].x, xv[u][1].x, xv[u][0].y, xv[u][1].y};
      const uint32_t f1[4] = {xv[u][0].z, xv[u][1].z, xv[u][0].w, xv[u][1].w};
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        mma_16816(acc[n], f0, w[u][n].x, w[u][n].y);
        mma_16816(acc[n], f1, w[u][n].z, w[u][n].w);
      }
    }
  }
  // the first columns of B and C of this warp, on their way while h is summed.  Column 8 q + 2 i + b of a
  // 32-wide group is column 2 q + b of product i: a lane owns eight consecutive columns of two rows.
  constexpr int NS = (NT + 1) / 2;  // 16-wide steps over the rank
  const __nv_bfloat16* wb = p.b + static_cast<size_t>(ad) * p.N * p.R;
  uint2 bv[4][NS];
  uint4 cv[2];
  auto fetch = [&](int gr) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = gr * 32 + (g >> 1) * 8 + 2 * i + (g & 1);
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        const int r = s * 16 + q * 4;
        bv[i][s] = gr < g1 && n < p.N && r < p.R
                       ? __ldg(reinterpret_cast<const uint2*>(wb + static_cast<size_t>(n) * p.R + r))
                       : make_uint2(0u, 0u);
      }
    }
    const int col = gr * 32 + q * 8;
    const bool in = gr < g1 && col < p.N;
    cv[0] = in && row0 >= 0 ? *reinterpret_cast<const uint4*>(p.C + static_cast<size_t>(row0) * p.N + col) : zero;
    cv[1] = in && row1 >= 0 ? *reinterpret_cast<const uint4*>(p.C + static_cast<size_t>(row1) * p.N + col) : zero;
  };
  fetch(g0 + warp);
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    float* part = s_part + warp * 16 * LD + n * 8 + q * 2;
    *reinterpret_cast<float2*>(part + g * LD) = make_float2(acc[n][0], acc[n][1]);
    *reinterpret_cast<float2*>(part + (g + 8) * LD) = make_float2(acc[n][2], acc[n][3]);
  }
  const float scale = p.scaling ? p.scaling[ad] : 1.0f;
  __syncthreads();
  for (int i = threadIdx.x; i < 16 * LD / 4; i += kLoraThreads) {  // (the rows' padding is summed along)
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int w = 0; w < kLoraWarps; ++w) {
      const float4 t = *reinterpret_cast<const float4*>(s_part + w * 16 * LD + i * 4);
      v = make_float4(v.x + t.x, v.y + t.y, v.z + t.z, v.w + t.w);
    }
    *reinterpret_cast<float4*>(s_part + i * 4) = v;
  }
  cluster_sync_all();
  const uint32_t part = smem_addr(s_part);
  for (int i = threadIdx.x; i < 16 * LD / 4; i += kLoraThreads) {
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int c = 0; c < CL; ++c) {
      const float4 w = ld_dsmem_f4(mapa_shared(part + i * 16, c));
      v = make_float4(v.x + w.x, v.y + w.y, v.z + w.z, v.w + w.w);
    }
    // ranks that only pad are 0 even where x (times the 0 of A) made a NaN of them
    *reinterpret_cast<float4*>(s_h + i * 4) =
        i * 4 % LD < p.R ? make_float4(v.x * scale, v.y * scale, v.z * scale, v.w * scale) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  }
  cluster_sync_all();  // every rank has read the parts; s_h is complete

  // delta = h B^T.  The three bf16 parts of h go through the tensor cores, so h keeps its 24 bits.
  uint32_t hp[kLoraParts][NS][4];
#pragma unroll
  for (int s = 0; s < NS; ++s) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {  // four ranks of rows g and g + 8; ranks past the padded one are 0
      const int r = s * 16 + q * 4;
      const float4 v = r < RP ? *reinterpret_cast<const float4*>(s_h + (g + i * 8) * LD + r)
                              : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      uint32_t xy[kLoraParts], zw[kLoraParts];
      split_bf16x2(v.x, v.y, xy);
      split_bf16x2(v.z, v.w, zw);
#pragma unroll
      for (int part = 0; part < kLoraParts; ++part) {
        hp[part][s][i] = xy[part];
        hp[part][s][i + 2] = zw[part];
      }
    }
  }
  for (int gr = g0 + warp; gr < g1; gr += kLoraWarps) {
    float d[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int c = 0; c < 4; ++c) d[i][c] = 0.0f;
#pragma unroll
      for (int s = 0; s < NS; ++s) {
#pragma unroll
        for (int part = 0; part < kLoraParts; ++part) mma_16816(d[i], hp[part][s], bv[i][s].x, bv[i][s].y);
      }
    }
    const uint4 c0 = cv[0], c1 = cv[1];
    fetch(gr + kLoraWarps);
    const int col = gr * 32 + q * 8;
    if (col >= p.N) continue;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int row = s ? row1 : row0;
      if (row < 0) continue;
      const uint32_t c[4] = {s ? c1.x : c0.x, s ? c1.y : c0.y, s ? c1.z : c0.z, s ? c1.w : c0.w};
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float(c[i] << 16) + d[i][2 * s],
                                                       __uint_as_float(c[i] & 0xFFFF0000u) + d[i][2 * s + 1]);
        o[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
      *reinterpret_cast<uint4*>(p.out + static_cast<size_t>(row) * p.N + col) = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

// ---------------------------------------------------------------------------- many rows
// Rows sorted by adapter, tiles of 128 of one adapter, both products on the tensor cores, in two kernels of
// two CTAs per SM (one above rank 64):
//   lora_down_kernel  parts of h = x A^T.  The (tile, 64 columns of K) units are split evenly over the CTAs, so that a
//                     few tiles more or less than SMs cost nothing; x gathered and A copied by cp.async into
//                     128-byte-swizzled tiles, tcgen05.mma into TMEM.
//   lora_up_kernel    out = C + h B^T, the (tile, 64 columns of N) units split the same way.  A CTA sums the parts of its
//                     tile's h in the order of K, scales it and keeps it in TMEM as three bf16 parts (all 24 bits),
//                     from where the products take it; C and B come by cp.async, the product goes into one of two
//                     TMEM buffers while the chunk before is added and stored.
// Bound by HBM: x once, C in and out; 4096 rows, rank 64, 7168 -> 4096: 52 us with the sort (one at a
// time, from cold caches: down 18.6 us for 66 MB, up 28 for 75).  mma.sync took 28 us for the second product of 4096 x
// 4096, rank 64, whose bytes take 11; parts summed once by the last CTA of a tile took 8 us, in every reader 3; h as two
// parts in shared memory, so 16 bits of it, 51 us in all.
constexpr int kLoraTileRows = 128;
constexpr uint64_t kLoraWaitNs = 2000000000ull;  // far above any legal wait
constexpr int kLoraTimeout = 6;                  // FG_ERR_TIMEOUT

template <int RP>
struct LoraTile {
  static constexpr int KB = (RP + 63) / 64;            // 64-wide blocks of the rank
  static constexpr int X_BYTES = kLoraTileRows * 128;  // 128 rows x 64 columns
  static constexpr int STAGE_BYTES = X_BYTES + RP * 128;
  static constexpr int CTAS = RP <= 64 ? 2 : 1;  // per SM
  static constexpr int STAGES = (CTAS == 2 ? 100 : 200) * 1024 / STAGE_BYTES;
  static constexpr int DOWN_SMEM = 1024 + STAGES * STAGE_BYTES;
  static constexpr int PART_FLOATS = kLoraTileRows * RP;
  static constexpr int B_BYTES = KB * 64 * 128;
  static constexpr int RING = RP <= 64 ? 3 : 4;  // chunks of C and B in shared memory
  static constexpr int UP_SMEM = 1024 + RING * (X_BYTES + B_BYTES);
  // TMEM of lora_up_kernel: two products of 64 columns, then the parts of h, two bf16 a column
  static constexpr int UP_H = 128, UP_PART = RP / 2;
  static constexpr int UP_TMEM = UP_H + kLoraParts * UP_PART <= 256 ? 256 : 512;
  static_assert(CTAS * UP_TMEM <= 512 && UP_H + kLoraParts * UP_PART <= UP_TMEM, "TMEM");
  static_assert(CTAS * (DOWN_SMEM + 1536) <= 227 * 1024 && CTAS * (UP_SMEM + 1536) <= 227 * 1024, "shared memory");
};

// Units [begin(c), begin(c + 1)) of U belong to CTA c of P; U >= P.
__device__ __forceinline__ int lora_begin(int c, int P, long long U) { return static_cast<int>(c * U / P); }
__device__ __forceinline__ int lora_owner(int u, int P, long long U) {
  return static_cast<int>(((static_cast<long long>(u) + 1) * P - 1) / U);
}

// 16 bytes global -> shared, zeros where `in` is false (the address must be valid all the same).
__device__ __forceinline__ void cp_async_16_or_zero(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ uint4 ld_shared_16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_shared_16(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
// D[tmem] (+)= A[smem desc] * B[smem desc]^T, bf16 operands, fp32 accumulator.
__device__ __forceinline__ void mma_bf16(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// The same with A in TMEM: lane m, two consecutive values of a row in each 32-bit column.
__device__ __forceinline__ void mma_bf16_tmem(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                              uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// 32 lanes x 4 consecutive 32-bit columns: thread t writes lane (base + t).
__device__ __forceinline__ void tmem_st_32x32b_x4(uint32_t taddr, const uint32_t (&r)[4]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3])
               : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// Instruction descriptor: bf16 x bf16 -> f32, both operands K-major, shape M x N.
__host__ __device__ constexpr uint32_t idesc_bf16_f32(int M, int N) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

// CTAs of lora_down_kernel's grid that have units: of U units, KB a tile, each takes at least about sqrt(3/4 KB).  A
// unit costs its CTA 0.4 us and a part of a tile's h its readers 0.3, so that a tile of KB units is best
// cut into about sqrt(4/3 KB) parts (KB = 3: 2, 112: 12) where there are CTAs enough.
__device__ __forceinline__ int lora_down_ctas(long long U, int KB, unsigned grid) {
  long long least = 1;
  while (4 * least * least < 3ll * KB) ++least;
  const long long most = (U + least - 1) / least;
  return static_cast<int>(most < grid ? most : grid);
}

// Rows of a tile that thread `tid` copies 16 bytes of: row_of + 32 i; -1 for padding.  (The places are read past
// L1: lora_up_kernel reads them before it has waited for lora_down_kernel.)
__device__ __forceinline__ void lora_tile_rows(const LoraParams& p, int tile, int row_of, int (&row)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int at = tile * kLoraTileRows + row_of + 32 * i;
    row[i] = __ldcg(p.group + at) >= 0 ? __ldcg(p.place_row + at) : -1;
  }
}

template <int RP>
__global__ void __launch_bounds__(kLoraThreads, LoraTile<RP>::CTAS) lora_down_kernel(const LoraParams p) {
  typedef LoraTile<RP> L;
  constexpr int STAGES = L::STAGES;
  constexpr uint32_t TMEM_COLS = RP < 32 ? 32 : RP;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t done[STAGES];
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
  // copies: 8 threads take the 128 bytes of a row, 32 rows at once
  const int piece = tid & 7, row_of = tid >> 3;
  const uint32_t swizzled = static_cast<uint32_t>(row_of * 128 + ((piece ^ (row_of & 7)) << 4));
  if (tid == 0) {
    for (int s = 0; s < STAGES; ++s) mbar_init(&done[s], 1);
    s_abort = 0;
    fence_mbar_init();
  }
  // before the next kernel may start: its CTAs take theirs early, and wait for this kernel with it
  if (warp == 0) {
    tmem_alloc(&s_tmem, TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  pdl_wait_prior_grid();
  pdl_launch_dependents();
  const int KB = (p.K + 63) / 64;
  const long long U = static_cast<long long>(p.tiles[0]) * KB;
  const int P = lora_down_ctas(U, KB, gridDim.x);
  if (static_cast<int>(blockIdx.x) >= P) {
    if (warp == 0) tmem_dealloc(tmem, TMEM_COLS);
    return;
  }
  const int u0 = lora_begin(blockIdx.x, P, U), n = lora_begin(blockIdx.x + 1, P, U) - u0;

  // the loads run ahead of the products, over the tiles: their own tile, place in K and ring
  int load_tile = u0 / KB, load_kb = u0 - load_tile * KB, load_stage = 0;
  const __nv_bfloat16 *xr[4], *wr[(RP + 31) / 32];
  bool has[4];
  auto load_rows = [&]() {
    int row[4];
    lora_tile_rows(p, load_tile, row_of, row);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      has[i] = row[i] >= 0;
      xr[i] = p.x + static_cast<size_t>(max(row[i], 0)) * p.K + piece * 8;
    }
    const __nv_bfloat16* wa = p.a + static_cast<size_t>(p.group[load_tile * kLoraTileRows]) * p.R * p.K + piece * 8;
#pragma unroll
    for (int i = 0; i < (RP + 31) / 32; ++i) wr[i] = wa + static_cast<size_t>(min(row_of + 32 * i, p.R - 1)) * p.K;
  };
  load_rows();
  auto load = [&]() {
    const bool in = load_kb * 64 + piece * 8 < p.K;
    const int at = in ? load_kb * 64 : -piece * 8;
    const uint32_t st = base + load_stage * L::STAGE_BYTES + swizzled;
#pragma unroll
    for (int i = 0; i < 4; ++i) cp_async_16_or_zero(st + i * 32 * 128, xr[i] + at, in && has[i]);
#pragma unroll
    for (int i = 0; i < (RP + 31) / 32; ++i) {
      const int r = row_of + 32 * i;
      if (RP % 32 == 0 || r < RP) cp_async_16_or_zero(st + L::X_BYTES + i * 32 * 128, wr[i] + at, in && r < p.R);
    }
    if (++load_stage == STAGES) load_stage = 0;
  };
  auto load_next = [&]() {  // the unit after the last one loaded
    if (++load_kb == KB) {
      load_kb = 0;
      ++load_tile;
      load_rows();
    }
    load();
  };
  bool ok = true;
  // (the test hook: no product has been issued, so this wait runs out)
  if (p.stall == 1 && tid == 0) ok = mbar_wait(&done[0], 0, &s_abort, kLoraWaitNs);
#pragma unroll 1
  for (int it = 0; it < STAGES - 1; ++it) {
    if (it == 0)
      load();
    else if (it < n)
      load_next();
    cp_async_commit();
  }
  int t = u0 / KB, kb = u0 - t * KB;
  bool fresh = true;  // the first unit of its tile here
#pragma unroll 1
  for (int it = 0; it < n; ++it) {
    cp_async_wait<STAGES - 2>();
    fence_proxy_async_smem();
    __syncthreads();
    if (tid == 0 && ok) {
      tc_fence_after();
      const uint32_t st = base + (it % STAGES) * L::STAGE_BYTES;
      const uint64_t adesc = smem_desc_k128_sw128(st), bdesc = smem_desc_k128_sw128(st + L::X_BYTES);
#pragma unroll
      for (int j = 0; j < 4; ++j)  // 16 values = 32 bytes = 2 descriptor units per step
        mma_bf16(tmem, adesc + 2 * j, bdesc + 2 * j, idesc_bf16_f32(kLoraTileRows, RP), !fresh || j > 0 ? 1u : 0u);
      mma_commit(&done[it % STAGES]);
    }
    const int next = it + STAGES - 1;
    if (next < n) {
      if (it > 0 && ok)  // the products that read this place of the ring
        ok = mbar_wait(&done[next % STAGES], ((it - 1) / STAGES) & 1u, &s_abort, kLoraWaitNs);
      if (ok) load_next();
    }
    cp_async_commit();
    fresh = false;
    if (kb < KB - 1 && it < n - 1) {
      ++kb;
      continue;
    }

    // the tile ends here, or this CTA's share of it does
    if (ok) ok = mbar_wait(&done[it % STAGES], (it / STAGES) & 1u, &s_abort, kLoraWaitNs);
    tc_fence_after();
    // a whole tile has a place of its own; of a CTA's two places for parts, the second is for the tile that
    // begins in it, the first for one that began in an earlier CTA
    const bool begins = t * KB >= u0, ends = kb == KB - 1;
    const int place = begins && ends ? 2 * gridDim.x + t : 2 * blockIdx.x + (begins ? 1 : 0);
    float4* part = reinterpret_cast<float4*>(p.parts + static_cast<size_t>(place) * L::PART_FLOATS);
    fresh = true;
    kb = 0;
    ++t;
    {
      constexpr int CPW = RP >= 32 ? RP / 2 : RP;
      constexpr int STEP = CPW < 32 ? 16 : 32;
      const int c0 = (warp >> 2) * CPW, m = (warp & 3) * 32 + lane;
      if (c0 < RP) {
#pragma unroll
        for (int c = 0; c < CPW; c += STEP) {
          uint32_t v[STEP];
          const uint32_t at = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + c0 + c;
          if constexpr (STEP == 16)
            tmem_ld_32x32b_x16(at, v);
          else
            tmem_ld_32x32b_x32(at, v);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < STEP; i += 4) {
            const uint32_t poison = s_abort ? 0x7fffffffu : 0u;  // NaN after a wait that ran out
            part[((c0 + c + i) / 4) * kLoraTileRows + m] =
                make_float4(__uint_as_float(v[i] | poison), __uint_as_float(v[i + 1] | poison),
                            __uint_as_float(v[i + 2] | poison), __uint_as_float(v[i + 3] | poison));
          }
        }
      }
    }
    tc_fence_before();  // the next tile's products come after the barrier at the top of the loop
  }
  cp_async_wait<0>();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, TMEM_COLS);
  if (s_abort && tid == 0) atomicCAS(p.status, 0, kLoraTimeout);
}

template <int RP>
__global__ void __launch_bounds__(kLoraThreads, LoraTile<RP>::CTAS) lora_up_kernel(const LoraParams p) {
  typedef LoraTile<RP> L;
  constexpr int RING = L::RING;
  constexpr uint32_t TMEM_COLS = L::UP_TMEM;
  constexpr uint32_t C_RING = 0, B_RING = C_RING + RING * L::X_BYTES;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t done[2];
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const int piece = tid & 7, row_of = tid >> 3;
  const uint32_t swizzled = static_cast<uint32_t>(row_of * 128 + ((piece ^ (row_of & 7)) << 4));
  if (tid == 0) {
    mbar_init(&done[0], 1);
    mbar_init(&done[1], 1);
    s_abort = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(&s_tmem, TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;

  // The preceding kernel, lora_down_kernel, let this one start after it had waited for all before it: only the
  // parts of h, and what is written, come after the wait below.
  const int chunks = (p.N + 63) / 64;
  const int KB = (p.K + 63) / 64;
  const long long U = static_cast<long long>(__ldcg(p.tiles)) * KB;
  const int PU = lora_down_ctas(U, KB, gridDim.x);  // the grid of lora_down_kernel, as large as this one
  const long long V = static_cast<long long>(__ldcg(p.tiles)) * chunks;
  const int P = static_cast<int>(V < gridDim.x ? V : gridDim.x);
  int v = 0, v_end = 0;
  if (static_cast<int>(blockIdx.x) < P) {
    v = lora_begin(blockIdx.x, P, V);
    v_end = lora_begin(blockIdx.x + 1, P, V);
  }
  int row[4];
  bool ok = true, waited = false;
  if (p.stall == 2 && tid == 0) ok = mbar_wait(&done[0], 0, &s_abort, kLoraWaitNs);  // as in lora_down_kernel
  int used = 0;  // products so far: the TMEM buffer and the phase of its barrier go by it
  while (v < v_end) {
    const int t = v / chunks, c0 = v - t * chunks;
    const int nc = min(chunks - c0, v_end - v);
    const int ad = __ldcg(p.group + t * kLoraTileRows);
    lora_tile_rows(p, t, row_of, row);
    const __nv_bfloat16* wb = p.b + static_cast<size_t>(ad) * p.N * p.R;
    auto load = [&](int c) {
      const int col = (c0 + c) * 64 + piece * 8;
      const uint32_t cs = base + C_RING + (c % RING) * L::X_BYTES + swizzled;
      if (col < p.N) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (row[i] >= 0) cp_async_16_or_zero(cs + i * 32 * 128, p.C + static_cast<size_t>(row[i]) * p.N + col, true);
      }
      const uint32_t bs = base + B_RING + (c % RING) * L::B_BYTES + swizzled;
#pragma unroll
      for (int b = 0; b < L::KB; ++b) {
        const int r = b * 64 + piece * 8;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int nn = (c0 + c) * 64 + row_of + 32 * i;
          const bool in = nn < p.N && r < p.R;
          if (r < RP)
            cp_async_16_or_zero(bs + b * (64 * 128) + i * 32 * 128, wb + (in ? static_cast<size_t>(nn) * p.R + r : 0), in);
        }
      }
    };
    auto finish = [&](int c) {  // the chunk's product is on its way to TMEM, its C in shared memory
      const int use = used + c;
      if (ok) ok = mbar_wait(&done[use & 1], (use >> 1) & 1u, &s_abort, kLoraWaitNs);
      tc_fence_after();
      const int m = (warp & 3) * 32 + lane, half = warp >> 2;
      uint32_t d[32];
      tmem_ld_32x32b_x32(tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + (use & 1) * 64 + half * 32, d);
      tmem_wait_ld();
      tc_fence_before();
      if (!ok) {  // NaN after a wait that ran out
#pragma unroll
        for (int i = 0; i < 32; ++i) d[i] = 0x7fffffffu;
      }
      const uint32_t cs = base + C_RING + (c % RING) * L::X_BYTES;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t at = cs + m * 128 + (((half * 4 + j) ^ (m & 7)) << 4);
        const uint4 w = ld_shared_16(at);
        const uint32_t in[4] = {w.x, w.y, w.z, w.w};
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const __nv_bfloat162 s =
              __floats2bfloat162_rn(__uint_as_float(in[i] << 16) + __uint_as_float(d[8 * j + 2 * i]),
                                    __uint_as_float(in[i] & 0xFFFF0000u) + __uint_as_float(d[8 * j + 2 * i + 1]));
          o[i] = *reinterpret_cast<const uint32_t*>(&s);
        }
        st_shared_16(at, make_uint4(o[0], o[1], o[2], o[3]));
      }
      __syncthreads();
      const int col = (c0 + c) * 64 + piece * 8;
      if (col < p.N) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (row[i] >= 0)
            *reinterpret_cast<uint4*>(p.out + static_cast<size_t>(row[i]) * p.N + col) =
                ld_shared_16(cs + swizzled + i * 32 * 128);
      }
    };
#pragma unroll 1
    for (int c = 0; c < RING - 1; ++c) {
      if (c < nc) load(c);
      cp_async_commit();
    }
    if (!waited) {
      waited = true;
      pdl_wait_prior_grid();
      pdl_launch_dependents();
    }
    {  // h (its last product of the tile before has run: every thread has waited for it)
      const int first = lora_owner(t * KB, PU, U), last = lora_owner(t * KB + KB - 1, PU, U);
      const float scale = p.scaling ? p.scaling[ad] : 1.0f;
      // a thread's row is its lane of TMEM; its quads of ranks lie side by side, half of the row's
      constexpr int EACH = RP / 8, SIDE = EACH < 8 ? EACH : 8;  // quads of a thread; at once
      const int m = tid % kLoraTileRows, q0 = tid / kLoraTileRows * EACH;
      const uint32_t to = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + L::UP_H;
#pragma unroll 1
      for (int e = 0; e < EACH; e += SIDE) {
        float4 h[SIDE];
#pragma unroll
        for (int i = 0; i < SIDE; ++i) h[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 2
        for (int c = first; c <= last; ++c) {
          const int place = first == last ? 2 * gridDim.x + t : 2 * c + (c == first ? 1 : 0);
          const float4* part = reinterpret_cast<const float4*>(p.parts + static_cast<size_t>(place) * L::PART_FLOATS) +
                               (q0 + e) * kLoraTileRows + m;
          float4 w[SIDE];
#pragma unroll
          for (int i = 0; i < SIDE; ++i) w[i] = __ldcg(part + i * kLoraTileRows);
#pragma unroll
          for (int i = 0; i < SIDE; ++i)
            h[i] = make_float4(h[i].x + w[i].x, h[i].y + w[i].y, h[i].z + w[i].z, h[i].w + w[i].w);
        }
#pragma unroll
        for (int i = 0; i < SIDE; i += 2) {
          uint32_t out[kLoraParts][4];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const bool pads = (q0 + e + i + k) * 4 >= p.R;  // padding, which infinities in x make NaN
            const float4 v = h[i + k];
            uint32_t xy[kLoraParts], zw[kLoraParts];
            split_bf16x2(pads ? 0.0f : v.x * scale, pads ? 0.0f : v.y * scale, xy);
            split_bf16x2(pads ? 0.0f : v.z * scale, pads ? 0.0f : v.w * scale, zw);
#pragma unroll
            for (int part = 0; part < kLoraParts; ++part) {
              out[part][2 * k] = xy[part];
              out[part][2 * k + 1] = zw[part];
            }
          }
#pragma unroll
          for (int part = 0; part < kLoraParts; ++part)
            tmem_st_32x32b_x4(to + part * L::UP_PART + 2 * (q0 + e + i), out[part]);
        }
      }
      tmem_wait_st();
      tc_fence_before();  // the products come after the barrier below
    }
#pragma unroll 1
    for (int c = 0; c < nc; ++c) {
      cp_async_wait<RING - 2>();
      fence_proxy_async_smem();
      __syncthreads();
      if (tid == 0 && ok) {
        tc_fence_after();
        const uint32_t d = tmem + ((used + c) & 1) * 64;
#pragma unroll
        for (int part = 0; part < kLoraParts; ++part) {
          const uint32_t h = tmem + L::UP_H + part * L::UP_PART;
#pragma unroll
          for (int b = 0; b < L::KB; ++b) {
            const uint64_t bdesc = smem_desc_k128_sw128(base + B_RING + (c % RING) * L::B_BYTES + b * (64 * 128));
#pragma unroll
            for (int j = 0; j < (RP < 64 ? RP / 16 : 4); ++j)  // 16 values are 8 columns of h
              mma_bf16_tmem(d, h + 32 * b + 8 * j, bdesc + 2 * j, idesc_bf16_f32(kLoraTileRows, 64),
                            part + b + j > 0 ? 1u : 0u);
          }
        }
        mma_commit(&done[(used + c) & 1]);
      }
      if (c > 0) finish(c - 1);
      // The ring's place of chunk c - 1: its product has run, and of its C this thread overwrites only what it
      // has itself just stored.
      if (c + RING - 1 < nc) load(c + RING - 1);
      cp_async_commit();
    }
    finish(nc - 1);
    used += nc;
    v += nc;
  }
  if (!waited) {
    pdl_wait_prior_grid();
    pdl_launch_dependents();
  }
  cp_async_wait<0>();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, TMEM_COLS);
  if (s_abort && tid == 0) atomicCAS(p.status, 0, kLoraTimeout);

  // rows without an adapter
  if (p.out == p.C) return;
  const int pieces = p.N / 8;
  const long long todo = static_cast<long long>(p.tiles[1] - p.tiles[0]) * kLoraTileRows * pieces;
  for (long long i = static_cast<long long>(blockIdx.x) * kLoraThreads + tid; i < todo;
       i += static_cast<long long>(gridDim.x) * kLoraThreads) {
    const int at = p.tiles[0] * kLoraTileRows + static_cast<int>(i / pieces);
    if (p.group[at] < 0) continue;
    const size_t src = static_cast<size_t>(p.place_row[at]) * p.N + (i % pieces) * 8;
    *reinterpret_cast<uint4*>(p.out + src) = *reinterpret_cast<const uint4*>(p.C + src);
  }
}

}  // namespace fg
