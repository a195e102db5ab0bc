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
  // tiles of rows sorted by adapter (lora_tiles_kernel): place -> adapter (L: none, -1: padding) and row
  const int* group;
  const int* place_row;
  int* status;
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

// ---------------------------------------------------------------------------- many rows
// Tiles of 128 rows of one adapter, one cluster of four CTAs each, both products on the tensor cores:
//   1. a rank forms its part of h = x A^T over a quarter of K: 64 columns a stage, the rows of x gathered and the
//      rows of A copied by cp.async into 128-byte-swizzled tiles, tcgen05.mma into TMEM;
//   2. the four parts are summed in rank order, each rank summing 32 rows over distributed shared memory
//      and handing them, scaled and split into two bf16 halves, to all four;
//   3. each rank adds h B^T to its quarter of the columns of C, 64 at a time: C and B by cp.async, the
//      product into one of two TMEM buffers, while the chunk before is added and stored.
// Bound by HBM (x, C in and out); two CTAs share an SM (ranks up to 64), so that one's phases overlap
// the other's and a few tiles more than SMs do not cost a second wave.  mma.sync for the second product
// measured 28 us of a 45 us tile where this takes the time of its bytes.
constexpr int kLoraTileRows = 128;
constexpr int kLoraTileCluster = 4;
constexpr int kLoraRing = 3;                     // chunks of C and B in shared memory
constexpr uint64_t kLoraWaitNs = 2000000000ull;  // far above any legal wait
constexpr int kLoraTimeout = 6;                  // FG_ERR_TIMEOUT

template <int RP>
struct LoraTile {
  static constexpr int LD = RP + 4;                     // row of a part of h, floats
  static constexpr int KB = (RP + 63) / 64;             // 64-wide blocks of the rank
  static constexpr int X_BYTES = kLoraTileRows * 128;   // 128 rows x 64 columns
  static constexpr int STAGES = RP <= 64 ? 4 : 5;
  static constexpr int STAGE_BYTES = X_BYTES + RP * 128;
  static constexpr int H_BYTES = KB * X_BYTES;          // one half of h
  static constexpr int PART = 2 * H_BYTES;              // offsets: the part of h; the rings
  static constexpr int C_RING = 2 * H_BYTES;
  static constexpr int B_RING = C_RING + kLoraRing * X_BYTES;
  static constexpr int B_BYTES = KB * 64 * 128;
  static constexpr int END = B_RING + kLoraRing * B_BYTES;
  static constexpr int SMEM = 1024 + (END > STAGES * STAGE_BYTES ? END : STAGES * STAGE_BYTES);
  static_assert(PART + kLoraTileRows * LD * 4 <= SMEM - 1024, "part of h");
  static_assert(SMEM <= 227 * 1024 && (RP > 64 || 2 * (SMEM + 2048) <= 227 * 1024), "shared memory");
};

// 16 bytes global -> shared, zeros where `in` is false (the address must be valid all the same).
__device__ __forceinline__ void cp_async_16_or_zero(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void st_dsmem_2(uint32_t cluster_addr, uint32_t a, uint32_t b) {
  asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};" ::"r"(cluster_addr), "r"(a), "r"(b) : "memory");
}
__device__ __forceinline__ uint4 ld_shared_16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_shared_16(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
// Orders generic-proxy writes to shared memory of the cluster before later accesses of the async proxy.
__device__ __forceinline__ void fence_proxy_async_all() { asm volatile("fence.proxy.async;" ::: "memory"); }
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
// Instruction descriptor: bf16 x bf16 -> f32, both operands K-major, shape M x N.
__host__ __device__ constexpr uint32_t idesc_bf16_f32(int M, int N) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

template <int RP>
__global__ void __launch_bounds__(kLoraThreads, RP <= 64 ? 2 : 1) lora_tiles_kernel(const LoraParams p) {
  typedef LoraTile<RP> L;
  constexpr int STAGES = L::STAGES;
  constexpr uint32_t TMEM_COLS = 128;
  extern __shared__ uint8_t smem_raw[];
  __shared__ int s_row[kLoraTileRows];
  __shared__ __align__(8) uint64_t done[STAGES];
  __shared__ __align__(8) uint64_t chunk_done[2];
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const int tile = blockIdx.x / kLoraTileCluster;
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;  // the same in every CTA of the cluster
  // copies: 8 threads take the 128 bytes of a row, 32 rows at once
  const int piece = tid & 7, row_of = tid >> 3;
  const uint32_t swizzled = static_cast<uint32_t>(row_of * 128 + ((piece ^ (row_of & 7)) << 4));

  pdl_wait_prior_grid();
  pdl_launch_dependents();
  const int ad = p.group[tile * kLoraTileRows];
  if (ad < 0 || (ad >= p.L && p.out == p.C)) return;  // the same for the whole cluster
  if (tid < kLoraTileRows) {
    const int at = tile * kLoraTileRows + tid;
    s_row[tid] = p.group[at] >= 0 ? p.place_row[at] : -1;
  }
  const int chunks = (p.N + 63) / 64;
  const int c0 = static_cast<int>(static_cast<long long>(chunks) * rank / kLoraTileCluster);
  const int nc = static_cast<int>(static_cast<long long>(chunks) * (rank + 1) / kLoraTileCluster) - c0;
  if (tid == 0) {
    for (int s = 0; s < STAGES; ++s) mbar_init(&done[s], 1);
    mbar_init(&chunk_done[0], 1);
    mbar_init(&chunk_done[1], 1);
    s_abort = 0;
    fence_mbar_init();
  }
  if (warp == 0 && ad < p.L) {
    tmem_alloc(&s_tmem, TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  int row[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) row[i] = s_row[row_of + 32 * i];
  if (ad >= p.L) {  // no adapter: the rows are copied
    for (int c = c0; c < c0 + nc; ++c) {
      const int col = c * 64 + piece * 8;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (row[i] < 0 || col >= p.N) continue;
        const size_t at = static_cast<size_t>(row[i]) * p.N + col;
        *reinterpret_cast<uint4*>(p.out + at) = *reinterpret_cast<const uint4*>(p.C + at);
      }
    }
    return;
  }
  const uint32_t tmem = s_tmem;

  // ---- 1. this rank's part of h
  const int kblocks = (p.K + 63) / 64;
  const int k0 = static_cast<int>(static_cast<long long>(kblocks) * rank / kLoraTileCluster);
  const int n = static_cast<int>(static_cast<long long>(kblocks) * (rank + 1) / kLoraTileCluster) - k0;
  const __nv_bfloat16* wa = p.a + static_cast<size_t>(ad) * p.R * p.K;
  auto load = [&](int it) {
    const int k = (k0 + it) * 64 + piece * 8;
    const bool in = k < p.K;
    const int at = in ? k : 0;
    const uint32_t st = base + (it % STAGES) * L::STAGE_BYTES + swizzled;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      cp_async_16_or_zero(st + i * 32 * 128, p.x + static_cast<size_t>(max(row[i], 0)) * p.K + at, in && row[i] >= 0);
#pragma unroll
    for (int i = 0; i < (RP + 31) / 32; ++i) {
      const int r = row_of + 32 * i;
      if (RP % 32 == 0 || r < RP)
        cp_async_16_or_zero(st + L::X_BYTES + i * 32 * 128, wa + static_cast<size_t>(r < p.R ? r : 0) * p.K + at,
                            in && r < p.R);
    }
  };
  bool ok = true;
#pragma unroll
  for (int it = 0; it < STAGES - 1; ++it) {
    if (it < n) load(it);
    cp_async_commit();
  }
  for (int it = 0; it < n; ++it) {
    cp_async_wait<STAGES - 2>();
    fence_proxy_async_smem();
    __syncthreads();
    if (tid == 0) {
      tc_fence_after();
      const uint32_t st = base + (it % STAGES) * L::STAGE_BYTES;
      const uint64_t adesc = smem_desc_k128_sw128(st), bdesc = smem_desc_k128_sw128(st + L::X_BYTES);
#pragma unroll
      for (int j = 0; j < 4; ++j)  // 16 values = 32 bytes = 2 descriptor units per step
        mma_bf16(tmem, adesc + 2 * j, bdesc + 2 * j, idesc_bf16_f32(kLoraTileRows, RP), it + j > 0 ? 1u : 0u);
      mma_commit(&done[it % STAGES]);
    }
    const int next = it + STAGES - 1;
    if (next < n) {
      if (it > 0 && ok)  // the products that read this slot
        ok = mbar_wait(&done[next % STAGES], ((it - 1) / STAGES) & 1u, &s_abort, kLoraWaitNs);
      if (ok) load(next);
    }
    cp_async_commit();
  }
  if (n > 0 && ok) ok = mbar_wait(&done[(n - 1) % STAGES], ((n - 1) / STAGES) & 1u, &s_abort, kLoraWaitNs);
  cp_async_wait<0>();
  __syncthreads();

  // ---- 2. the parts' sum; a warp reads lane quadrant warp % 4, the columns split between the warp halves
  tc_fence_after();
  float* s_part = reinterpret_cast<float*>(smem_raw + (base - raw) + L::PART);
  {
    constexpr int CPW = RP >= 32 ? RP / 2 : RP;
    constexpr int STEP = CPW < 32 ? 16 : 32;
    const int first = (warp >> 2) * CPW;
    float* dst = s_part + ((warp & 3) * 32 + lane) * L::LD;
    if (first < RP) {
#pragma unroll
      for (int c = 0; c < CPW; c += STEP) {
        uint32_t v[STEP];
        if (n > 0) {
          const uint32_t at = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + first + c;
          if constexpr (STEP == 16)
            tmem_ld_32x32b_x16(at, v);
          else
            tmem_ld_32x32b_x32(at, v);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int i = 0; i < STEP; ++i) v[i] = 0u;
        }
#pragma unroll
        for (int i = 0; i < STEP; i += 4)
          *reinterpret_cast<uint4*>(dst + first + c + i) = make_uint4(v[i], v[i + 1], v[i + 2], v[i + 3]);
      }
    }
  }
  tc_fence_before();
  cluster_sync_all();
  {
    const float scale = s_abort ? __int_as_float(0x7fffffff) : p.scaling ? p.scaling[ad] : 1.0f;
    constexpr int ROWS = kLoraTileRows / kLoraTileCluster;
    for (int i = tid; i < ROWS * RP / 4; i += kLoraThreads) {
      const int m = rank * ROWS + i / (RP / 4), r = i % (RP / 4) * 4;
      const uint32_t part = smem_addr(s_part + m * L::LD + r);
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int c = 0; c < kLoraTileCluster; ++c) {
        const float4 w = ld_dsmem_f4(mapa_shared(part, c));
        v = make_float4(v.x + w.x, v.y + w.y, v.z + w.z, v.w + w.w);
      }
      uint32_t hi[2], lo[2];
      split_bf16x2(v.x * scale, v.y * scale, hi[0], lo[0]);
      split_bf16x2(v.z * scale, v.w * scale, hi[1], lo[1]);
      const uint32_t at = base + (r / 64) * L::X_BYTES + m * 128 + (((r % 64) / 8 ^ (m & 7)) << 4) + (r & 4) * 2;
#pragma unroll
      for (int c = 0; c < kLoraTileCluster; ++c) {
        st_dsmem_2(mapa_shared(at, c), hi[0], hi[1]);
        st_dsmem_2(mapa_shared(at + L::H_BYTES, c), lo[0], lo[1]);
      }
    }
  }
  fence_proxy_async_all();
  cluster_sync_all();  // h is complete everywhere, and nobody touches another CTA's memory any more
  fence_proxy_async_all();

  // ---- 3. out = C + h B^T on this rank's columns
  const __nv_bfloat16* wb = p.b + static_cast<size_t>(ad) * p.N * p.R;
  auto load_chunk = [&](int c) {
    const int col = (c0 + c) * 64 + piece * 8;
    const uint32_t cs = base + L::C_RING + (c % kLoraRing) * L::X_BYTES + swizzled;
    if (col < p.N) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (row[i] >= 0) cp_async_16_or_zero(cs + i * 32 * 128, p.C + static_cast<size_t>(row[i]) * p.N + col, true);
    }
    const uint32_t bs = base + L::B_RING + (c % kLoraRing) * L::B_BYTES + swizzled;
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
  auto finish_chunk = [&](int c) {  // the chunk's product is in TMEM, its C in shared memory
    if (ok) ok = mbar_wait(&chunk_done[c & 1], (c >> 1) & 1u, &s_abort, kLoraWaitNs);
    tc_fence_after();
    const int m = (warp & 3) * 32 + lane, half = warp >> 2;
    uint32_t d[32];
    tmem_ld_32x32b_x32(tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + (c & 1) * 64 + half * 32, d);
    tmem_wait_ld();
    tc_fence_before();
    const uint32_t cs = base + L::C_RING + (c % kLoraRing) * L::X_BYTES;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t at = cs + m * 128 + (((half * 4 + j) ^ (m & 7)) << 4);
      const uint4 v = ld_shared_16(at);
      const uint32_t in[4] = {v.x, v.y, v.z, v.w};
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 t =
            __floats2bfloat162_rn(__uint_as_float(in[i] << 16) + __uint_as_float(d[8 * j + 2 * i]),
                                  __uint_as_float(in[i] & 0xFFFF0000u) + __uint_as_float(d[8 * j + 2 * i + 1]));
        o[i] = *reinterpret_cast<const uint32_t*>(&t);
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
  for (int c = 0; c < 2; ++c) {
    if (c < nc) load_chunk(c);
    cp_async_commit();
  }
#pragma unroll 1
  for (int c = 0; c < nc; ++c) {
    cp_async_wait<1>();
    fence_proxy_async_smem();
    __syncthreads();
    if (tid == 0) {
      tc_fence_after();
      const uint32_t d = tmem + (c & 1) * 64;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
#pragma unroll
        for (int b = 0; b < L::KB; ++b) {
          const uint64_t adesc = smem_desc_k128_sw128(base + half * L::H_BYTES + b * L::X_BYTES);
          const uint64_t bdesc =
              smem_desc_k128_sw128(base + L::B_RING + (c % kLoraRing) * L::B_BYTES + b * (64 * 128));
#pragma unroll
          for (int j = 0; j < (RP < 64 ? RP / 16 : 4); ++j)
            mma_bf16(d, adesc + 2 * j, bdesc + 2 * j, idesc_bf16_f32(kLoraTileRows, 64), half + b + j > 0 ? 1u : 0u);
        }
      }
      mma_commit(&chunk_done[c & 1]);
    }
    if (c > 0) finish_chunk(c - 1);
    // The ring's place of chunk c - 1: its product has run, and of its C this thread overwrites only what it
    // has itself just stored.
    if (c + 2 < nc) load_chunk(c + 2);
    cp_async_commit();
  }
  if (nc > 0) finish_chunk(nc - 1);
  cp_async_wait<0>();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, TMEM_COLS);
  if (s_abort && tid == 0) atomicCAS(p.status, 0, kLoraTimeout);
}

}  // namespace fg
