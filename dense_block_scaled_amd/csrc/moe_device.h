// moe_device.h -- what the mixture-of-experts kernels share on the device.
#pragma once

#include <hip/hip_runtime.h>

namespace dbs {

// Between LDS writes of a wave's lanes and other lanes' reads of them, or reads
// and the writes that follow.  The hardware keeps a wave's LDS operations in
// order; the fences keep the compiler from answering a read with what the
// lane itself had stored, or moving it (the barrier alone is one of scheduling).
// No instruction comes of it.
__device__ __forceinline__ void wave_handover()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

}  // namespace dbs
