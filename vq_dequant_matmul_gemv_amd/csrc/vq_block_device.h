// vq_block_device.h -- device code that the kernels of the operators around the
// products share.
#pragma once

#include "vq_device.h"

namespace vqmi {

// One wave's LDS writes before its later reads of other lanes' values (LDS
// runs a wave's accesses in order: only the compiler is held back).
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

}  // namespace vqmi
