// A barrier for what passes through LDS only: __syncthreads would also wait for every global load and store in flight, and
// with it for operands that are loaded ahead.  gfx950 only.
#pragma once

#include <hip/hip_runtime.h>

namespace bimamba {

__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

}  // namespace bimamba
