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

// The parts of s = 1 / (1 + e^-g) and of 1 - s as factors that stay normal
// numbers where s itself would not (g below -87, where silu(g) u need not be
// small): with h = e^(-|g| / 2) and r = 1 / (1 + h^2),
//
//     g >= 0:  s = r,      1 - s = h^2 r          g < 0:  s = h^2 r,  1 - s = r
//
// so s = p^2 r with p = 1 or h: p is multiplied into each of two factors.
struct Sigmoid {
    float p, r, rest;         // s = p p r; rest = 1 - s
};

__device__ __forceinline__ Sigmoid sigmoid(float g)
{
    const float h = __builtin_amdgcn_exp2f(fabsf(g) * -0.72134752f);     // log2(e) / 2
    const float e = h * h, r = __builtin_amdgcn_rcpf(1.0f + e);
    return g >= 0.0f ? Sigmoid{1.0f, r, e * r} : Sigmoid{h, r, r};
}

// silu(g) u
__device__ __forceinline__ float gated(float g, float u)
{
    const Sigmoid s = sigmoid(g);
    return g * s.p * s.r * (u * s.p);
}

}  // namespace dbs
