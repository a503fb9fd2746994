// operators.cuh -- building blocks of the kernels around the layer (norm.cu,
// router_bwd.cu) beside those of common.cuh.
#pragma once

#include "common.cuh"

namespace moe {

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
