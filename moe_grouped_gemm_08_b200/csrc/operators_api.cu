// operators_api.cu -- host side of the operators around the GEMMs (the router, the experts' row
// layout, dispatch, combine, low-rank adapters): argument checks and launches.  Nothing here
// allocates, reads device memory or synchronises, so every call can be captured into a CUDA graph;
// none needs fg_init.
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <cstring>
#include <type_traits>

#include "fp8gemm.h"
#include "lora_kernels.cuh"
#include "moe_route_kernels.cuh"
#include "moe_rows_kernels.cuh"

namespace {

constexpr int kMaxDevices = 64;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

long long cdiv(long long a, long long b) { return (a + b - 1) / b; }

int sm_count() {
  static std::atomic<int> cached[kMaxDevices];
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
    cudaGetLastError();
    return 0;
  }
  int v = cached[dev].load(std::memory_order_relaxed);
  if (v > 0) return v;
  if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || v <= 0) {
    cudaGetLastError();
    return 0;
  }
  cached[dev].store(v, std::memory_order_relaxed);
  return v;
}

// Programmatic dependent launch, as the GEMMs are launched: every kernel here waits for the preceding
// grid before it lets the next one start, and before it touches global memory.  lora_up_kernel alone reads earlier
// what the grid before it, which has waited for all others, does not write.
template <typename... Params, typename... Args>
fg_status launch(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, void* stream, int cluster,
                 const Args&... args) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  if (cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...) != cudaSuccess) {
    cudaGetLastError();
    return FG_ERR_CUDA;
  }
  return FG_OK;
}

// CTAs of a kernel that the device holds at once: the grid of a kernel whose CTAs walk over their work
// (more would run as a second, mostly empty wave).  0 if the device cannot be asked.
template <auto KERNEL>
long long resident_ctas(int threads) {
  static std::atomic<int> cached[kMaxDevices];
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
  int n = cached[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, KERNEL, threads, 0) != cudaSuccess || n <= 0) {
      cudaGetLastError();
      return 0;
    }
    cached[dev].store(n, std::memory_order_relaxed);
  }
  return static_cast<long long>(n) * sm_count();
}

// Launch with one CTA per `work` unit, `waves` times as many at most as the device holds at once.
template <auto KERNEL, int waves = 1, typename... Args>
fg_status launch_walk(long long work, int threads, void* stream, const Args&... args) {
  const long long most = waves * resident_ctas<KERNEL>(threads);
  if (most <= 0) return FG_ERR_CUDA;
  return launch(KERNEL, dim3(static_cast<unsigned>(work < most ? work : most)), threads, 0, stream, 1, args...);
}

// The opt-in shared-memory size of a kernel, set once per device (not again during a capture).
template <auto KERNEL>
bool allow_smem(size_t bytes) {
  static std::atomic<uint64_t> done{0};
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return false;
  const uint64_t bit = 1ull << dev;
  if (done.load(std::memory_order_acquire) & bit) return true;
  if (cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes)) !=
      cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  done.fetch_or(bit, std::memory_order_acq_rel);
  return true;
}

// ------------------------------------------------------------------------------------ the router
size_t value_bytes(int dtype) { return dtype == FG_F32 ? 4 : 2; }
bool valid_dtype(int dtype) { return dtype == FG_F32 || dtype == FG_BF16 || dtype == FG_F16; }

// Lanes that hold a row of E columns, and the rows that a CTA's warps take at once.
int route_step(int E) { return fg::kRouteWarps * (E <= 64 ? 4 : E <= 128 ? 2 : 1); }

// How a sequence of T rows is split over CTAs.  Up to four rows a warp of eight CTAs: one cluster per
// sequence, which also finishes (one launch).  Otherwise a second kernel finishes, and the chunks are such that
// every SM gets about eight CTAs where that leaves them three rows a warp, else four (32768 rows of 256
// experts: 28.9 us with eight, 31.7 with four; 8192 rows: 16.3 and 14.1, as the chunks have to be summed).
struct RouteSplit {
  int rows, chunks;  // rows per CTA, CTAs per sequence
  bool cluster;
};
RouteSplit route_split(int S, int T, int E, int sms) {
  RouteSplit r;
  const int step = route_step(E);
  r.cluster = E <= fg::kRouteThreads && T <= 4 * fg::kRouteMaxCluster * step;
  const long long all = static_cast<long long>(S) * T, ctas = all >= 3ll * step * 8 * sms ? 8ll * sms : 4ll * sms;
  const long long share = r.cluster ? cdiv(T, fg::kRouteMaxCluster) : cdiv(all, ctas);
  const long long rows = cdiv(share, step) * step;
  r.rows = static_cast<int>(rows < T ? rows : T);
  r.chunks = static_cast<int>(cdiv(T, r.rows));
  return r;
}

template <typename T, int LPR, int NPL, int V>
fg_status route_launch(const fg::RouteParams& p, int S, bool cluster, void* stream) {
  if constexpr (LPR * NPL <= fg::kRouteThreads) {
    if (cluster)
      return launch(fg::moe_route_kernel<T, LPR, NPL, V, true>, dim3(p.chunks, S), fg::kRouteThreads, 0, stream,
                    p.chunks, p);
  }
  return launch(fg::moe_route_kernel<T, LPR, NPL, V, false>, dim3(p.chunks, S), fg::kRouteThreads, 0, stream, 1, p);
}
template <typename T, int LPR, int NPL, int V>
fg_status route_launch(const fg::RouteGradParams& p, int S, bool, void* stream) {
  return launch(fg::moe_route_backward_kernel<T, LPR, NPL, V>, dim3(static_cast<unsigned>(cdiv(p.T, p.rows_per_chunk)), S),
                fg::kRouteThreads, 0, stream, 1, p);
}

// The instance that holds E columns: few lanes a row for few experts, 16-byte loads where each row
// starts on a 16-byte boundary.
template <typename T, typename P>
fg_status route_pick(const P& p, int S, bool cluster, bool wide, void* stream) {
  constexpr int V = 16 / static_cast<int>(sizeof(T));
  const int E = p.E;
  if (wide) {
    if (E <= 64) return route_launch<T, 8, 8, V>(p, S, cluster, stream);
    if (E <= 128) return route_launch<T, 16, 8, V>(p, S, cluster, stream);
    if (E <= 256) return route_launch<T, 32, 8, V>(p, S, cluster, stream);
    if (E <= 512) return route_launch<T, 32, 16, V>(p, S, cluster, stream);
    return route_launch<T, 32, 32, V>(p, S, cluster, stream);
  }
  if (E <= 8) return route_launch<T, 8, 1, 1>(p, S, cluster, stream);
  if (E <= 32) return route_launch<T, 8, 4, 1>(p, S, cluster, stream);
  if (E <= 64) return route_launch<T, 8, 8, 1>(p, S, cluster, stream);
  if (E <= 128) return route_launch<T, 16, 8, 1>(p, S, cluster, stream);
  if (E <= 256) return route_launch<T, 32, 8, 1>(p, S, cluster, stream);
  if (E <= 512) return route_launch<T, 32, 16, 1>(p, S, cluster, stream);
  return route_launch<T, 32, 32, 1>(p, S, cluster, stream);
}

template <typename P>
fg_status route_dispatch(const P& p, int S, int dtype, bool cluster, bool wide, void* stream) {
  if (dtype == FG_F32) return route_pick<float>(p, S, cluster, wide, stream);
  if (dtype == FG_BF16) return route_pick<__nv_bfloat16>(p, S, cluster, wide, stream);
  return route_pick<__half>(p, S, cluster, wide, stream);
}

fg_status route_check(int dtype, int S, int T, int E, int k) {
  if (!valid_dtype(dtype) || S < 0 || T < 0 || E <= 0 || k <= 0 || k > E) return FG_ERR_INVALID_ARG;
  if (E > FG_MOE_MAX_EXPERTS || k > fg::kRouteMaxK || S > 65535) return FG_ERR_UNSUPPORTED;
  return FG_OK;
}

size_t route_part_bytes(int S, int E, const RouteSplit& r) { return static_cast<size_t>(S) * r.chunks * E * 4; }
size_t route_scratch_bytes(int S, int E, const RouteSplit& r) {
  if (r.cluster) return 0;
  return route_part_bytes(S, E, r) + static_cast<size_t>(S) * r.chunks * (E + 1) * 4;
}

// ------------------------------------------------------------------------------------ row layouts
// How the pairs are split: one chunk (and one launch) up to 2048, then 512 a chunk while that leaves a CTA per
// SM or fewer, then 2048, and 8192 above a million, as every CTA reads all chunks' counts.  (4096 pairs of 8
// experts: 4.7 us in eight chunks, 5.9 us in one.)
struct LayoutSplit {
  int threads, items;
};
LayoutSplit layout_split(long long pairs) {
  if (pairs <= 512) return {256, 2};
  if (pairs <= 2048) return {1024, 2};
  if (pairs <= 148 * 512) return {256, 2};
  if (pairs <= 512 * 2048) return {256, 8};
  return {1024, 8};
}
int layout_chunks(long long pairs) {
  const LayoutSplit s = layout_split(pairs);
  return static_cast<int>(cdiv(pairs, static_cast<long long>(s.threads) * s.items));
}

template <int THREADS, int ITEMS>
fg_status layout_launch(const fg::LayoutParams& p, void* stream) {
  constexpr size_t most = THREADS / 32 * fg::kLayoutMaxExperts * 2;
  const size_t smem = static_cast<size_t>(THREADS / 32) * p.E * 2;
  if (!allow_smem<fg::moe_layout_kernel<THREADS, ITEMS>>(most)) return FG_ERR_CUDA;
  if constexpr (THREADS * ITEMS != 2048 || THREADS != 1024) {  // that split has one chunk
    if (p.chunks > 1) {
      const fg_status s = launch(fg::moe_layout_count_kernel<THREADS, ITEMS>, dim3(p.chunks), THREADS, 0, stream, 1, p);
      if (s != FG_OK) return s;
    }
  }
  // a CTA per chunk, and one per 4096 rows of m_indices up to 128 (256 experts, 512 pairs: 51 us with one CTA)
  long long ctas = cdiv(p.M, 4096);
  if (ctas > 128) ctas = 128;
  if (ctas < p.chunks) ctas = p.chunks;
  if (ctas < 1) ctas = 1;
  return launch(fg::moe_layout_kernel<THREADS, ITEMS>, dim3(static_cast<unsigned>(ctas)), THREADS, smem, stream, 1, p);
}

size_t layout_hist_bytes(long long pairs, int E) {
  const int chunks = layout_chunks(pairs);
  return chunks > 1 ? static_cast<size_t>(chunks) * E * 4 : 0;
}

fg_status layout_run(fg::LayoutParams& p, void* stream) {
  p.chunks = layout_chunks(p.pairs);
  const LayoutSplit s = layout_split(p.pairs);
  if (s.threads == 1024) return s.items == 2 ? layout_launch<1024, 2>(p, stream) : layout_launch<1024, 8>(p, stream);
  return s.items == 2 ? layout_launch<256, 2>(p, stream) : layout_launch<256, 8>(p, stream);
}

fg_status layout_call(const int* ids, int* rows, int* group, long long pairs, int E, int M, int mmax, void* scratch,
                      size_t scratch_bytes, void* stream) {
  const size_t need = layout_hist_bytes(pairs, E);
  if (need > 0 && (!scratch || scratch_bytes < need)) return FG_ERR_INVALID_ARG;
  if (!aligned(scratch, 4)) return FG_ERR_ALIGNMENT;
  fg::LayoutParams p;
  std::memset(&p, 0, sizeof(p));
  p.ids = ids;
  p.rows = rows;
  p.group = group;
  p.hist = static_cast<int*>(scratch);
  p.pairs = pairs;
  p.E = E;
  p.M = M;
  p.mmax = mmax;
  p.align = fg_m_alignment();
  return layout_run(p, stream);
}

fg_status layout_check(const int* ids, const int* rows, const int* group, long long pairs, int E) {
  if (pairs < 0 || E <= 0 || !group || (pairs > 0 && (!ids || !rows))) return FG_ERR_INVALID_ARG;
  if (E > FG_MOE_MAX_EXPERTS || pairs > (1ll << 24)) return FG_ERR_UNSUPPORTED;
  if (!aligned(ids, 4) || !aligned(rows, 4) || !aligned(group, 4)) return FG_ERR_ALIGNMENT;
  return FG_OK;
}

template <int NT, int CL>
fg_status lora_rows_launch(const fg::LoraParams& p, void* stream) {
  constexpr size_t smem = fg::LoraRows<NT>::SMEM;
  if (!allow_smem<fg::lora_rows_kernel<NT, CL>>(smem)) return FG_ERR_CUDA;
  return launch(fg::lora_rows_kernel<NT, CL>, dim3(static_cast<unsigned>(p.M) * CL), fg::kLoraThreads, smem, stream, CL, p);
}

// Eight CTAs a cluster up to 64 rows, else four.  With eight, then four, K 7168, N 4096: 64 rows of 64 adapters 8.9 and
// 11.3 us at rank 16 (31.1 and 23.0 at rank 64, 60.8 and 57.2 at rank 128, where fewer CTAs fit at once), of 8
// adapters 6.9 and 8.4, 13.5 and 16.0, 17.8 and 23.9; 128 rows of 64 adapters 15.0 and 12.5, 34.7 and 24.9,
// 83.5 and 61.7, of 8 adapters 7.7 and 8.6, 14.8 and 17.4, 26.4 and 26.9.
template <int NT>
fg_status lora_rows_pick(const fg::LoraParams& p, void* stream) {
  return p.M <= 64 ? lora_rows_launch<NT, 8>(p, stream) : lora_rows_launch<NT, 4>(p, stream);
}

template <int RP>
fg_status lora_tiles_launch(const fg::LoraParams& p, int sms, void* stream) {
  typedef fg::LoraTile<RP> L;
  if (!allow_smem<fg::lora_down_kernel<RP>>(L::DOWN_SMEM) || !allow_smem<fg::lora_up_kernel<RP>>(L::UP_SMEM))
    return FG_ERR_CUDA;
  const dim3 grid(static_cast<unsigned>(sms * L::CTAS));
  const fg_status s = launch(fg::lora_down_kernel<RP>, grid, fg::kLoraThreads, L::DOWN_SMEM, stream, 1, p);
  if (s != FG_OK) return s;
  return launch(fg::lora_up_kernel<RP>, grid, fg::kLoraThreads, L::UP_SMEM, stream, 1, p);
}

// Many rows: tiles of 128 rows, sorted by adapter.  Few, or more adapters than the sort takes: groups of 16, which the
// kernel finds by reading all rows' adapters, so that its time grows with the square of the rows (hence
// kMostUnsortedRows).  Tiles, then groups, K 7168, N 4096: 300 rows of 8 adapters 19.2 and 12.0 us at rank 16, 25.2 and
// 21.5 at rank 64, 36.2 and 36.6 at rank 128; 512 rows 19.5 and 14.7, 24.9 and 27.9, 36.9 and 55.9; 1000 rows 23.4
// and 25.2, 32.6 and 45.9, 41.9 and 90.2.  (Of 64 adapters, half empty tiles: 300 rows 45 and 15, 55 and 35, 93 and 83;
// 1000 rows 47 and 29, 56 and 57, 96 and 119.)
bool lora_by_tiles(int M, int L) { return L > 0 && L < FG_MOE_MAX_EXPERTS && M > 256; }
constexpr int kMostUnsortedRows = 1 << 18;

// Scratch of the tiles: parts of h, then the places of the sorted rows (of the L adapters and of those without).
struct LoraScratch {
  int places, tiles;
  size_t group, hist, bytes;
};
LoraScratch lora_scratch(int M, int L, int R, int sms) {
  LoraScratch s;
  const int n = M < L + 1 ? M : L + 1;
  s.tiles = n + (M - n) / fg::kLoraTileRows;
  s.places = s.tiles * fg::kLoraTileRows;
  const size_t rank = R <= 16 ? 16 : R <= 32 ? 32 : R <= 64 ? 64 : 128;
  const int ctas = sms * (rank <= 64 ? fg::LoraTile<64>::CTAS : fg::LoraTile<128>::CTAS);
  s.group = static_cast<size_t>(2 * ctas + s.tiles) * fg::kLoraTileRows * rank * 4;
  s.hist = s.group + static_cast<size_t>(s.places) * 8 + 8;
  s.bytes = s.hist + layout_hist_bytes(M, L + 1);
  return s;
}

std::atomic<int> g_lora_stall{0};  // fg_lora_debug_set_stall

__device__ int g_lora_status;  // FG_ERR_TIMEOUT once a wait of the kernels for many rows has run out

// Its address, looked up once per device (not again during a capture).
int* lora_status_word() {
  static std::atomic<int*> cached[kMaxDevices];
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
    cudaGetLastError();
    return nullptr;
  }
  int* at = cached[dev].load(std::memory_order_acquire);
  if (at) return at;
  void* v = nullptr;
  if (cudaGetSymbolAddress(&v, g_lora_status) != cudaSuccess) {
    cudaGetLastError();
    return nullptr;
  }
  cached[dev].store(static_cast<int*>(v), std::memory_order_release);
  return static_cast<int*>(v);
}

}  // namespace

extern "C" {


size_t fg_moe_route_scratch_bytes(int S, int T, int E) {
  if (S <= 0 || T <= 0 || E <= 0) return 0;
  const int sms = sm_count();
  return sms > 0 ? route_scratch_bytes(S, E, route_split(S, T, E, sms)) : 0;
}

fg_status fg_moe_route(const void* logits, int dtype, const unsigned char* mask, int* ids, float* weights, int* counts,
                       float* loss, float* slope, int S, int T, int E, int k, int renormalize, void* scratch,
                       size_t scratch_bytes, void* stream) {
  const fg_status bad = route_check(dtype, S, T, E, k);
  if (bad != FG_OK) return bad;
  if (S == 0) return FG_OK;
  if (!counts || !loss || !slope || (T > 0 && (!logits || !ids || !weights))) return FG_ERR_INVALID_ARG;
  if (!aligned(logits, value_bytes(dtype)) || !aligned(ids, 4) || !aligned(weights, 4) || !aligned(counts, 4) ||
      !aligned(loss, 4) || !aligned(slope, 4) || !aligned(scratch, 4))
    return FG_ERR_ALIGNMENT;
  const int sms = sm_count();
  if (sms <= 0) return FG_ERR_CUDA;
  fg::RouteParams p;
  std::memset(&p, 0, sizeof(p));
  p.logits = logits;
  p.mask = mask;
  p.ids = ids;
  p.weights = weights;
  p.counts = counts;
  p.loss = loss;
  p.slope = slope;
  p.T = T;
  p.E = E;
  p.k = k;
  p.renorm = renormalize ? 1 : 0;
  if (T > 0) {
    const RouteSplit r = route_split(S, T, E, sms);
    const size_t need = route_scratch_bytes(S, E, r);
    if (need > 0 && (!scratch || scratch_bytes < need)) return FG_ERR_INVALID_ARG;
    p.part_p = static_cast<float*>(scratch);
    p.part_n = need > 0 ? reinterpret_cast<int*>(static_cast<char*>(scratch) + route_part_bytes(S, E, r)) : nullptr;
    p.chunks = r.chunks;
    p.rows_per_chunk = r.rows;
    const bool wide = aligned(logits, 16) && static_cast<size_t>(E) * value_bytes(dtype) % 16 == 0;
    const fg_status s = route_dispatch(p, S, dtype, r.cluster, wide, stream);
    if (s != FG_OK || r.cluster) return s;
  }
  return launch(fg::moe_route_finish_kernel, dim3(fg::kFinishCluster, S), 1024, 0, stream, fg::kFinishCluster, p);
}

fg_status fg_moe_route_backward(const void* logits, int dtype, const int* ids, const float* slope,
                                const float* grad_weights, const float* grad_loss, void* grad_logits, int S, int T,
                                int E, int k, int renormalize, void* stream) {
  const fg_status bad = route_check(dtype, S, T, E, k);
  if (bad != FG_OK) return bad;
  if (S == 0 || T == 0) return FG_OK;
  if (!logits || !ids || !slope || !grad_logits) return FG_ERR_INVALID_ARG;
  const size_t size = value_bytes(dtype);
  if (!aligned(logits, size) || !aligned(grad_logits, size) || !aligned(ids, 4) || !aligned(slope, 4) ||
      !aligned(grad_weights, 4) || !aligned(grad_loss, 4))
    return FG_ERR_ALIGNMENT;
  const int sms = sm_count();
  if (sms <= 0) return FG_ERR_CUDA;
  fg::RouteGradParams p;
  p.logits = logits;
  p.ids = ids;
  p.slope = slope;
  p.grad_weights = grad_weights;
  p.grad_loss = grad_loss;
  p.grad_logits = grad_logits;
  p.T = T;
  p.E = E;
  p.k = k;
  const int step = route_step(E);
  p.rows_per_chunk = static_cast<int>(cdiv(cdiv(static_cast<long long>(S) * T, 4ll * sms), step) * step);
  p.renorm = renormalize ? 1 : 0;
  const bool wide = aligned(logits, 16) && aligned(grad_logits, 16) && static_cast<size_t>(E) * size % 16 == 0;
  return route_dispatch(p, S, dtype, false, wide, stream);
}

long long fg_moe_layout_rows(long long pairs, int E) {
  if (pairs <= 0 || E <= 0) return 0;
  const long long n = pairs < E ? pairs : E;  // experts with rows
  return fg_m_alignment() * (n + (pairs - n) / fg_m_alignment());
}

size_t fg_moe_layout_scratch_bytes(long long pairs, int E) {
  if (pairs <= 0 || E <= 0 || pairs > (1ll << 24)) return 0;
  return layout_hist_bytes(pairs, E);
}

fg_status fg_moe_layout_contiguous(const int* ids, int* rows, int* m_indices, long long pairs, int E, int M,
                                   void* scratch, size_t scratch_bytes, void* stream) {
  if (pairs == 0 && M == 0 && E > 0) return FG_OK;
  const fg_status s = layout_check(ids, rows, m_indices, pairs, E);
  if (s != FG_OK) return s;
  if (M < fg_moe_layout_rows(pairs, E)) return FG_ERR_INVALID_ARG;
  return layout_call(ids, rows, m_indices, pairs, E, M, 0, scratch, scratch_bytes, stream);
}

fg_status fg_moe_layout_masked(const int* ids, int* rows, int* masked_m, long long pairs, int E, int mmax,
                               void* scratch, size_t scratch_bytes, void* stream) {
  const fg_status s = layout_check(ids, rows, masked_m, pairs, E);
  if (s != FG_OK) return s;
  if (mmax <= 0) return FG_ERR_INVALID_ARG;
  if (static_cast<long long>(E) * mmax > 0x7fffffffll) return FG_ERR_UNSUPPORTED;
  return layout_call(ids, rows, masked_m, pairs, E, 0, mmax, scratch, scratch_bytes, stream);
}

fg_status fg_moe_dispatch_fp8(const void* x, const int* rows, void* A, float* sfa, int T, int k, int G, int M, int K,
                              int fmt, void* stream) {
  if (T < 0 || k < 0 || G < 0 || M < 0 || K < 0 || (fmt != FG_E4M3 && fmt != FG_E5M2)) return FG_ERR_INVALID_ARG;
  if (T == 0 || k == 0 || G == 0 || M == 0 || K == 0) return FG_OK;
  if (!x || !rows || !A || !sfa) return FG_ERR_INVALID_ARG;
  if (K % 16 != 0 || !aligned(x, 16) || !aligned(A, 16) || !aligned(sfa, 4) || !aligned(rows, 4))
    return FG_ERR_ALIGNMENT;
  if (k > fg::kRowsMaxK || static_cast<long long>(G) * M > 0x7fffffffll || M > FG_MOE_MAX_ROWS) return FG_ERR_UNSUPPORTED;
  fg::DispatchParams p;
  p.x = static_cast<const __nv_bfloat16*>(x);
  p.rows = rows;
  p.A = static_cast<uint8_t*>(A);
  p.sfa = sfa;
  p.T = T;
  p.k = k;
  p.K = K;
  p.M = G * M;
  p.mmax = M;
  p.ld = fg_sfa_ld(M);
  const int chunks = static_cast<int>(cdiv(K, 512 * fg::kDispatchSpans));
  const long long blocks = cdiv(static_cast<long long>(T) * chunks, 8);
  // eight short waves: CTAs that end at different times leave less idle than one long walk each (16384
  // tokens of 7168 columns: 82 us, one wave 94 us)
  return fmt == FG_E4M3 ? launch_walk<fg::moe_dispatch_kernel<0>, 8>(blocks, 256, stream, p, chunks)
                        : launch_walk<fg::moe_dispatch_kernel<1>, 8>(blocks, 256, stream, p, chunks);
}

static fg_status combine_check(int T, int k, int M, int N) {
  if (T < 0 || k < 0 || M < 0 || N < 0) return FG_ERR_INVALID_ARG;
  if (N % 8 != 0) return FG_ERR_ALIGNMENT;
  if (k > fg::kRowsMaxK) return FG_ERR_UNSUPPORTED;
  return FG_OK;
}

fg_status fg_moe_combine(const void* C, const int* rows, const float* weights, void* out, int T, int k, int M, int N,
                         void* stream) {
  const fg_status bad = combine_check(T, k, M, N);
  if (bad != FG_OK) return bad;
  if (T == 0 || N == 0) return FG_OK;
  if (!out || (k > 0 && (!rows || (M > 0 && !C)))) return FG_ERR_INVALID_ARG;
  if (!aligned(C, 16) || !aligned(out, 16) || !aligned(rows, 4) || !aligned(weights, 4)) return FG_ERR_ALIGNMENT;
  fg::CombineParams p;
  p.C = static_cast<const __nv_bfloat16*>(C);
  p.rows = rows;
  p.weights = weights;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.T = T;
  p.k = k;
  p.N = N;
  p.M = M;
  auto run = [&](auto choices) {  // so many choices at once
    constexpr int J = decltype(choices)::value;
    const int chunks = static_cast<int>(cdiv(N, 8 / J * 256));
    return launch_walk<fg::moe_combine_kernel<J>>(cdiv(static_cast<long long>(T) * chunks, 8), 256, stream, p, chunks);
  };
  if (k <= 2) return run(std::integral_constant<int, 2>());
  return run(std::integral_constant<int, 4>());
}

fg_status fg_moe_combine_backward(const void* grad_out, const void* C, const int* rows, const float* weights,
                                  void* grad_C, float* grad_weights, int T, int k, int M, int N, void* stream) {
  const fg_status bad = combine_check(T, k, M, N);
  if (bad != FG_OK) return bad;
  if (T == 0 || k == 0) return FG_OK;
  if (!rows || !weights || !grad_weights || (N > 0 && (!grad_out || (M > 0 && (!C || !grad_C)))))
    return FG_ERR_INVALID_ARG;
  if (!aligned(grad_out, 16) || !aligned(C, 16) || !aligned(grad_C, 16) || !aligned(rows, 4) || !aligned(weights, 4) ||
      !aligned(grad_weights, 4))
    return FG_ERR_ALIGNMENT;
  fg::CombineGradParams p;
  p.grad_out = static_cast<const __nv_bfloat16*>(grad_out);
  p.C = static_cast<const __nv_bfloat16*>(C);
  p.rows = rows;
  p.weights = weights;
  p.grad_C = static_cast<__nv_bfloat16*>(grad_C);
  p.grad_weights = grad_weights;
  p.T = T;
  p.k = k;
  p.N = N;
  p.M = M;
  const long long tokens = T;
  if (k <= 2) return launch_walk<fg::moe_combine_backward_kernel<2>>(tokens, fg::kCombineGradThreads, stream, p);
  if (k <= 4) return launch_walk<fg::moe_combine_backward_kernel<4>>(tokens, fg::kCombineGradThreads, stream, p);
  return launch_walk<fg::moe_combine_backward_kernel<8>>(tokens * cdiv(k, 8), fg::kCombineGradThreads, stream, p);
}

size_t fg_lora_scratch_bytes(int M, int R, int L) {
  if (M <= 0 || R <= 0 || L <= 0 || R > fg::kLoraMaxRank || !lora_by_tiles(M, L)) return 0;
  const int sms = sm_count();
  return sms > 0 ? lora_scratch(M, L, R, sms).bytes : 0;
}

fg_status fg_lora_add(const void* C, const void* x, const void* lora_a, const void* lora_b, const int* adapters,
                      const float* scaling, void* out, int M, int N, int K, int R, int L, void* scratch,
                      size_t scratch_bytes, void* stream) {
  if (M < 0 || N < 0 || K < 0 || R < 0 || L < 0) return FG_ERR_INVALID_ARG;
  if (K % 16 != 0 || N % 8 != 0 || R % 8 != 0) return FG_ERR_ALIGNMENT;
  if (R > fg::kLoraMaxRank || M > (1 << 24)) return FG_ERR_UNSUPPORTED;
  if (M == 0 || N == 0) return FG_OK;
  if (!C || !out || !adapters) return FG_ERR_INVALID_ARG;
  if (K == 0 || R == 0) L = 0;  // no adapter adds anything
  if (L > 0 && (!x || !lora_a || !lora_b)) return FG_ERR_INVALID_ARG;
  if (!aligned(C, 16) || !aligned(x, 16) || !aligned(lora_a, 16) || !aligned(lora_b, 16) || !aligned(out, 16) ||
      !aligned(adapters, 4) || !aligned(scaling, 4) || !aligned(scratch, 16))
    return FG_ERR_ALIGNMENT;
  if (L >= FG_MOE_MAX_EXPERTS && M > kMostUnsortedRows) return FG_ERR_UNSUPPORTED;
  if (L == 0) {
    if (out != C && cudaMemcpyAsync(out, C, static_cast<size_t>(M) * N * 2, cudaMemcpyDeviceToDevice,
                                    static_cast<cudaStream_t>(stream)) != cudaSuccess) {
      cudaGetLastError();
      return FG_ERR_CUDA;
    }
    return FG_OK;
  }
  fg::LoraParams p;
  std::memset(&p, 0, sizeof(p));
  p.C = static_cast<const __nv_bfloat16*>(C);
  p.x = static_cast<const __nv_bfloat16*>(x);
  p.a = static_cast<const __nv_bfloat16*>(lora_a);
  p.b = static_cast<const __nv_bfloat16*>(lora_b);
  p.adapters = adapters;
  p.scaling = scaling;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.M = M;
  p.N = N;
  p.K = K;
  p.R = R;
  p.L = L;
  if (lora_by_tiles(M, L)) {
    const int sms = sm_count();
    if (sms <= 0) return FG_ERR_CUDA;
    const LoraScratch need = lora_scratch(M, L, R, sms);
    if (!scratch || scratch_bytes < need.bytes) return FG_ERR_INVALID_ARG;
    p.stall = g_lora_stall.load(std::memory_order_relaxed);
    p.status = lora_status_word();
    if (!p.status) return FG_ERR_CUDA;
    uint8_t* at = static_cast<uint8_t*>(scratch);
    fg::LayoutParams lp;
    std::memset(&lp, 0, sizeof(lp));
    lp.ids = adapters;
    lp.group = reinterpret_cast<int*>(at + need.group);
    lp.inverse = lp.group + need.places;
    lp.tiles = lp.inverse + need.places;
    lp.hist = reinterpret_cast<int*>(at + need.hist);
    lp.pairs = M;
    lp.E = L + 1;
    lp.M = need.places;
    lp.align = fg::kLoraTileRows;
    lp.rest = 1;
    p.group = lp.group;
    p.place_row = lp.inverse;
    p.tiles = lp.tiles;
    p.parts = reinterpret_cast<float*>(at);
    const fg_status s = layout_run(lp, stream);
    if (s != FG_OK) return s;
    if (R <= 16) return lora_tiles_launch<16>(p, sms, stream);
    if (R <= 32) return lora_tiles_launch<32>(p, sms, stream);
    if (R <= 64) return lora_tiles_launch<64>(p, sms, stream);
    return lora_tiles_launch<128>(p, sms, stream);
  }
  if (R <= 8) return lora_rows_pick<1>(p, stream);
  if (R <= 16) return lora_rows_pick<2>(p, stream);
  if (R <= 32) return lora_rows_pick<4>(p, stream);
  if (R <= 64) return lora_rows_pick<8>(p, stream);
  return lora_rows_pick<16>(p, stream);
}

int fg_lora_debug_set_stall(int kernel) { return g_lora_stall.exchange(kernel == 1 || kernel == 2 ? kernel : 0); }

fg_status fg_lora_status(void* stream) {
  int* at = lora_status_word();
  if (!at) return FG_ERR_CUDA;
  int v = 0;
  if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess ||
      cudaMemcpy(&v, at, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess ||
      (v != 0 && cudaMemset(at, 0, sizeof(int)) != cudaSuccess)) {
    cudaGetLastError();
    return FG_ERR_CUDA;
  }
  return static_cast<fg_status>(v);
}

}  // extern "C"
