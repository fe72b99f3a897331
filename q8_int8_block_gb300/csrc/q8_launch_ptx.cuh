// q8_launch_ptx.cuh -- what kernels of attention over a cache share beyond q8_attn_ptx.cuh: dependent
// launches, the block cluster, pairs of bfloat16.
#pragma once
#include <cstdint>

#include <cuda_bf16.h>

#include "q8_ptx.cuh"

namespace q8 {

// two values rounded to bfloat16, lo in the low half
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Launches that depend on the kernel in front of them: that they may begin, and their wait for its end.
__device__ __forceinline__ void pdl_launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// The block cluster: a barrier of all its threads, and a value in the shared memory of CTA `rank`.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
__device__ __forceinline__ float peer_load(const float* own, int rank) {
  uint32_t at;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(own)), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
  return v;
}

}  // namespace q8
