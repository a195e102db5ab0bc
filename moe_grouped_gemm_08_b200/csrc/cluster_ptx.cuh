// cluster_ptx.cuh -- loads from the shared memory of the CTAs of a cluster.
#pragma once

#include <cstdint>

namespace fg {

// A 32-bit word of the shared memory of a CTA of the cluster (a shared::cluster address).
__device__ __forceinline__ float ld_dsmem_f32(uint32_t cluster_addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(cluster_addr) : "memory");
  return v;
}

}  // namespace fg
