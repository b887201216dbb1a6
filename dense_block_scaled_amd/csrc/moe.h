// moe.h -- internal interface between the C ABI of the mixture-of-experts
// operators (moe.cpp) and their gfx950 kernels (moe_route.hip, moe_gemm.hip,
// moe_pointwise.hip).  Not installed; callers use include/dbs.h.
#pragma once

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

namespace dbs {

constexpr int kMoeMaxExperts = 1024;
constexpr int kMoeMaxK = 16;             // experts per token: one lane of a 16-lane token group each
constexpr int kRouteTokens = 64;         // tokens per workgroup of the routing kernels (bits of a mask word)

// The expert products.  Group g owns rows offsets[g] .. offsets[g+1]-1 of the
// sorted order; offsets are read on the device and clamped to 0 .. M there.
struct MoeGemm {
    const uint8_t *X;         // T x K bf16 (gathered through rows) or M x K (rows null)
    const uint8_t *W;         // E x N x K bf16 (K-major) or E x K x N (MN-major)
    uint8_t *D;               // M x ncols bf16
    const int32_t *offsets;   // E + 1
    const int32_t *rows;      // M, or null
    int64_t T;                // rows of X
    int M, E, N, K;
    int ncols;                // columns of D: N, or N / 2 behind the gate
    int gate;                 // 1: D = silu(first N/2 columns) * last N/2 columns
    int wmn;                  // 1: W MN-major
    int vec;                  // 1 if D rows take 16-byte stores (ncols % 8 == 0, D 16-byte aligned)
};

// dW_g = dY_g^T X_g: N x K per expert, summed over the group's rows.
struct MoeGemmDw {
    const uint8_t *dY;        // M x N bf16
    const uint8_t *X;         // T x K bf16 (gathered) or M x K
    uint8_t *dW;              // E x N x K, bf16 or fp32
    const int32_t *offsets, *rows;
    int64_t T;
    int M, E, N, K;
    int f32;                  // 1: dW holds fp32
    int accumulate;           // 1: add to dW (fp32 only)
};

// Rows of an output tile (64, 128 or 256) for M rows over E experts on `cus`
// compute units, by the time of the busiest one (the rule and what it rests
// on: moe.cpp).
int moe_tile_rows(int64_t M, int64_t E, int64_t N, int64_t ncols, bool wmn, bool gate, int cus);

// Whether dW of `groups` experts is computed in 64 x 128 tiles (else 256 x 256)
// by `wgs` workgroups: the longest group's stages (64 rows), and the sums of
// all groups' with at least two and four to a group (what it rests on: at
// moe_dw in moe_gemm.hip).
__host__ __device__ inline bool moe_dw_small(int groups, int longest, int two, int four, int N, int K, bool f32, int wgs)
{
    const float many = (float)(((N + 255) / 256) * ((K + 255) / 256)) / (float)wgs;    // tiles of a group a workgroup
    const float few = (float)(((N + 63) / 64) * ((K + 127) / 128)) / (float)wgs;
    const float large = (f32 ? 90.0f : 50.0f) * ceilf(many * groups) + fmaxf(13.0f * longest, 16.0f * many * two);
    const float little = 10.0f * ceilf(few * groups) + fmaxf(3.5f * longest, 5.0f * few * four);
    return little < large;
}

// rows: 64, 128 or 256 per output tile
hipError_t launch_moe_tiles(const MoeGemm &p, int rows, int cus, hipStream_t stream);
hipError_t launch_moe_dw(const MoeGemmDw &p, int cus, hipStream_t stream);
// workgroups of moe_dw
int moe_dw_grid(int64_t E, int64_t N, int64_t K, int cus);

struct MoeRoute {
    const void *logits;       // T x E, fp32 or bf16
    int bf16;
    int64_t T;
    int E, k, renorm;
    int32_t *experts;         // T x k
    float *weights;           // T x k
    int32_t *offsets;         // E + 1
    int32_t *rows;            // T k
    int32_t *slots;           // T x k
    int32_t *counts;          // workspace: one row of E per kRouteTokens tokens, then E totals
};
int64_t moe_route_workspace_bytes(int64_t T, int64_t E);
hipError_t launch_moe_route(const MoeRoute &p, hipStream_t stream);
hipError_t launch_moe_route_bwd(const void *logits, int bf16, int64_t T, int E, int k, int renorm,
                                const int32_t *experts, const float *dweights, void *dlogits, hipStream_t stream);

hipError_t launch_swiglu(const void *H, void *A, int64_t M, int64_t F, hipStream_t stream);
hipError_t launch_swiglu_bwd(const void *dA, const void *H, void *dH, int64_t M, int64_t F, hipStream_t stream);
hipError_t launch_moe_combine(const void *Y, const int32_t *slots, const float *weights, void *out, int64_t T,
                              int64_t M, int k, int64_t H, hipStream_t stream);
hipError_t launch_moe_combine_bwd(const void *dO, const void *Y, const int32_t *slots, const float *weights,
                                  const int32_t *total, void *dY, float *dweights, int64_t T, int64_t M, int k,
                                  int64_t H, hipStream_t stream);

// Compute units of the current device, cached (dbs.cpp); a dbs_status, with
// the error text recorded.
int device_compute_units(int *cus);

}  // namespace dbs

// For the tests that say which kernel a size reaches (not in include/dbs.h):
// the rules above; stages: each expert's number of 64-row stages.
extern "C" int dbs_moe_tile_rows(int64_t M, int64_t E, int64_t N, int wmn, int gate, int cus);
extern "C" int dbs_moe_dw_small(const int32_t *stages, int E, int N, int K, int f32, int accumulate, int cus);
