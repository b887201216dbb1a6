// i8.cpp -- the C ABI of the 8-bit integer operators declared in include/dbs.h:
// argument validation, choice of kernel and launch.
#include "i8.h"

#include <hip/hip_runtime.h>

#include <cstdio>

#include "dbs.h"
#include "launch.h"
#include "moe.h"

namespace {

dbs_status fail(dbs_status st, const char *msg)
{
    dbs::set_error(msg);
    return st;
}

dbs_status done(hipError_t e)
{
    if (e == hipSuccess) return DBS_OK;
    char text[256];
    std::snprintf(text, sizeof(text), "kernel launch: %s", hipGetErrorString(e));
    return fail(DBS_EHIP, text);
}

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

constexpr int64_t kMaxRows = int64_t(1) << 25;
constexpr int64_t kMaxWidth = int64_t(1) << 21;     // N; K of the quantiser
constexpr int64_t kMaxK = (int64_t(1) << 17) - 1;   // of a product: 2^14 K stays below 2^31
constexpr int64_t kGatherLimit = 0xFF000000;        // bytes of a gathered X
constexpr int64_t kTwoGiB = int64_t(1) << 31;
constexpr int64_t kMostTiles = int64_t(1) << 30;

dbs_status check_product(const void *X, const float *sX, const void *W, const float *sW, const void *D, int64_t T,
                         int64_t M, int64_t E, int64_t N, int64_t K)
{
    if (!X || !sX || !W || !sW || !D) return fail(DBS_EINVAL, "null pointer argument");
    if (T <= 0 || M <= 0 || E <= 0 || N <= 0 || K <= 0) return fail(DBS_EINVAL, "sizes must be positive");
    if (T > kMaxRows || M > kMaxRows) return fail(DBS_EINVAL, "more than 2^25 rows");
    if (E > dbs::kMoeMaxExperts) return fail(DBS_EINVAL, "more than 1024 experts");
    if (N > kMaxWidth) return fail(DBS_EINVAL, "N above 2^21");
    if (K % 16) return fail(DBS_EINVAL, "K must be a multiple of 16");
    if (K > kMaxK) return fail(DBS_EINVAL, "K above 131056: sums could leave 32 bits");
    if (!aligned(X, 16) || !aligned(W, 16)) return fail(DBS_EINVAL, "codes must be 16-byte aligned");
    if (!aligned(sX, 4) || !aligned(sW, 4)) return fail(DBS_EINVAL, "scales must be 4-byte aligned");
    return DBS_OK;
}

dbs::I8Gemm product(const void *X, const float *sX, const void *W, const float *sW, void *D, int64_t T, int64_t M,
                    int64_t E, int64_t N, int64_t K)
{
    dbs::I8Gemm p{};
    p.X = static_cast<const uint8_t *>(X);
    p.W = static_cast<const uint8_t *>(W);
    p.sX = sX;
    p.sW = sW;
    p.D = static_cast<uint8_t *>(D);
    p.T = T;
    p.M = (int)M;
    p.E = (int)E;
    p.N = (int)N;
    p.K = (int)K;
    p.ncols = (int)N;
    return p;
}

dbs_status run_product(dbs::I8Gemm p, hipStream_t stream)
{
    // the kernels number their tiles (64 x 32 the smallest) in int, with a round of workgroups to spare
    if (((int64_t)p.M / 64 + p.E) * (((int64_t)p.ncols + 31) / 32) >= kMostTiles)
        return fail(DBS_EUNSUPPORTED, "too many output tiles");
    int cus = 0;
    const int st = dbs::device_compute_units(&cus);
    if (st != DBS_OK) return (dbs_status)st;
    p.vec = p.ncols % (p.f32 ? 4 : 8) == 0 && aligned(p.D, 16);
    const int height = dbs::moe_tile_rows(p.M, p.E, p.N, p.ncols, false, p.gate, cus);
    return done(dbs::launch_i8_tiles(p, height, cus, stream));
}

// What the experts' products check beyond check_product.
dbs_status check_sorted(const void *D, const int32_t *offsets, const int32_t *rows, int64_t T, int64_t M, int64_t K)
{
    if (!offsets) return fail(DBS_EINVAL, "null pointer argument");
    if (!rows && T != M) return fail(DBS_EINVAL, "without row indices X must have M rows");
    if (!aligned(D, 2)) return fail(DBS_EINVAL, "the output must be 2-byte aligned");
    if (!aligned(offsets, 4) || (rows && !aligned(rows, 4)))
        return fail(DBS_EINVAL, "offsets and rows must be 4-byte aligned");
    if (rows && T * K > kGatherLimit) return fail(DBS_EUNSUPPORTED, "a gathered X of nearly 4 GiB or more");
    return DBS_OK;
}

}  // namespace

extern "C" {

dbs_status quant_i8(dbs_real type, const void *x, int64_t M, int64_t K, int8_t *codes, float *scales, hipStream_t stream)
{
    if (!x || !codes || !scales) return fail(DBS_EINVAL, "null pointer argument");
    if (type != DBS_F32 && type != DBS_BF16) return fail(DBS_EINVAL, "unknown input type");
    if (M <= 0 || K <= 0) return fail(DBS_EINVAL, "sizes must be positive");
    if (M > kMaxRows || K > kMaxWidth) return fail(DBS_EINVAL, "rows above 2^25 or width above 2^21");
    if (!aligned(x, type == DBS_F32 ? 4 : 2) || !aligned(scales, 4)) return fail(DBS_EINVAL, "misaligned array");
    return done(dbs::launch_quant_i8(x, type == DBS_BF16, M, K, codes, scales, stream));
}

dbs_status gemm_i8(dbs_real type, const void *A, const float *sA, const void *B, const float *sB, void *D, int64_t M,
                   int64_t N, int64_t K, hipStream_t stream)
{
    dbs_status st = check_product(A, sA, B, sB, D, M, M, 1, N, K);
    if (st != DBS_OK) return st;
    if (type != DBS_F32 && type != DBS_BF16) return fail(DBS_EINVAL, "unknown output type");
    if (!aligned(D, type == DBS_F32 ? 4 : 2)) return fail(DBS_EINVAL, "misaligned output");
    dbs::I8Gemm p = product(A, sA, B, sB, D, M, M, 1, N, K);
    p.f32 = type == DBS_F32;
    return run_product(p, stream);
}

dbs_status gemm_moe_i8(const void *X, const float *sX, const void *W, const float *sW, void *D, const int32_t *offsets,
                       const int32_t *rows, int64_t T, int64_t M, int64_t E, int64_t N, int64_t K, hipStream_t stream)
{
    dbs_status st = check_product(X, sX, W, sW, D, T, M, E, N, K);
    if (st != DBS_OK) return st;
    if ((st = check_sorted(D, offsets, rows, T, M, K)) != DBS_OK) return st;
    dbs::I8Gemm p = product(X, sX, W, sW, D, T, M, E, N, K);
    p.offsets = offsets;
    p.rows = rows;
    return run_product(p, stream);
}

dbs_status gemm_moe_swiglu_i8(const void *X, const float *sX, const void *W, const float *sW, void *D,
                              const int32_t *offsets, const int32_t *rows, int64_t T, int64_t M, int64_t E, int64_t F,
                              int64_t K, hipStream_t stream)
{
    if (F > kMaxWidth / 2) return fail(DBS_EINVAL, "F above 2^20");
    dbs_status st = check_product(X, sX, W, sW, D, T, M, E, 2 * F, K);
    if (st != DBS_OK) return st;
    if ((st = check_sorted(D, offsets, rows, T, M, K)) != DBS_OK) return st;
    if (2 * F * K >= kTwoGiB) return fail(DBS_EUNSUPPORTED, "an expert's matrices of 2 GiB or more");
    dbs::I8Gemm p = product(X, sX, W, sW, D, T, M, E, 2 * F, K);
    p.offsets = offsets;
    p.rows = rows;
    p.ncols = (int)F;
    p.gate = 1;
    return run_product(p, stream);
}

}  // extern "C"
