// pool_add.cuh -- sums into a weights pool.
#pragma once

#include "common.cuh"

namespace sa {

// One token's weight: set, or added to.  (An addition without a read: the pool's old
// value need not come to the multiprocessor, and a page that two sequences share
// loses neither's.)
__device__ __forceinline__ void pool_put(float* at, float w, bool add) {
  if (add) asm volatile("red.relaxed.gpu.global.add.f32 [%0], %1;" ::"l"(at), "f"(w) : "memory");
  else *at = w;
}
// Four tokens', added (16-byte aligned).
__device__ __forceinline__ void pool_add4(float* at, float4 w) {
  asm volatile("red.relaxed.gpu.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(at), "f"(w.x), "f"(w.y), "f"(w.z),
               "f"(w.w)
               : "memory");
}

}  // namespace sa
