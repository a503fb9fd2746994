// operators.cuh -- building blocks of the kernels around the layer (norm.cu,
// router_bwd.cu) beside those of common.cuh.
#pragma once

#include <utility>

#include "common.cuh"

namespace moe {

// Kernels of one call that follow each other on a stream start early
// (programmatic dependent launch): a kernel lets its successor begin while it
// still runs (dependents_start), and a kernel launched by launch_next waits,
// behind its own set-up, until its predecessor is complete and its writes are
// visible (predecessor_done: before any access to memory that another kernel
// writes or reads).  What the predecessor writes changes while such a kernel is
// under way: its pointers are never const __restrict__ (read-only for a kernel's
// lifetime), and __ldg does not read them.  Worth about 2 us an edge.
__device__ __forceinline__ void dependents_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void predecessor_done() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename... P, typename... A>
inline cudaError_t launch_next(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, A &&...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
}

// Eight consecutive floats, one 32-byte sector (p 32-byte aligned).
__device__ __forceinline__ void st_f32x8(float *p, const float *v) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]),
               "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}

}  // namespace moe

namespace moe_host {
// Any rank up to 5: dims, strides (bytes, rank - 1 of them) and box innermost
// first; 128-byte swizzle, zeros out of bounds.
int encode_tmap(CUtensorMap *map, CUtensorMapDataType dtype, const void *base, int rank, const uint64_t *dims,
                const uint64_t *strides, const uint32_t *box);
}  // namespace moe_host
