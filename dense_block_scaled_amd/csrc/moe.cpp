// moe.cpp -- the C ABI of the mixture-of-experts operators declared in
// include/dbs.h: argument validation, choice of kernel and launch.
#include "moe.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdio>

#include "dbs.h"
#include "launch.h"

namespace dbs {

// Tiles of 64, 128 or 256 rows, by the time of the busiest CU in stages of a
// 256-row tile (1.3 us), for groups of M / E rows on average (half a tile
// of each is waste; few rows leave some experts without any).  A stage
// takes 0.22 of that (64 rows, K-major), 0.39 (MN-major, twice as wide), 0.85
// (128 rows), and reads W at the memory's rate, one of 256 rows of it per
// CU; large tiles come in whole rounds over the CUs, small ones even out.
// us with 64 / 128 / 256 rows: 8 experts of 4096 x 4096, 512 rows in all
// 56 / 66 / 69, 8192 rows 531 / 313 / 250; 8 of 1408 x 2048, 4096 rows 54 / 39 /
// 50; one of 2048 x 4096, 2048 rows 70 / 68 / 84; 128 of 1536 x 4096 behind the
// gate, 192 rows on 49 experts 123 / 152 / 156, 1536 rows on all 291 / 268 / 271;
// MN-major 18 of 776 x 2840, 4096 rows 43 / 55 / 68, 8192 rows 78 / 97 / 71.
int moe_tile_rows(int64_t M, int64_t E, int64_t N, int64_t ncols, bool wmn, bool gate, int cus)
{
    const int64_t likely = (2 * M * E + 2 * M + E - 1) / (2 * M + E), met = std::min(M, likely);
    auto per_cu = [&](int64_t tm, int64_t tn) {
        const int64_t rows = std::max(M / tm + met / 2, met);
        return double(rows * ((ncols + tn - 1) / tn)) / cus;
    };
    const double w = double(met) * N / 256 / cus;
    auto rounds = [&](int64_t tm, double stage) {
        const double n = per_cu(tm, gate ? 128 : 256), full = std::floor(n);
        return full * std::max(stage, w / n) + (n > full ? stage : 0.0);
    };
    const double t64 = std::max((wmn ? 0.39 : 0.22) * per_cu(64, wmn ? 128 : gate ? 32 : 64), 1.1 * w);
    const double t128 = rounds(128, 0.85), t256 = rounds(256, 1.0);
    return t64 <= t128 && t64 <= t256 ? 64 : t128 < t256 ? 128 : 256;
}

int moe_dw_grid(int64_t E, int64_t N, int64_t K, int cus)
{
    const int64_t tiles = E * ((N + 63) / 64) * ((K + 127) / 128);      // small ones: the more
    return (int)std::min<int64_t>(tiles, cus);
}

}  // namespace dbs

extern "C" int dbs_moe_tile_rows(int64_t M, int64_t E, int64_t N, int wmn, int gate, int cus)
{
    return dbs::moe_tile_rows(M, E, N, gate ? N / 2 : N, wmn, gate, cus);
}

extern "C" int dbs_moe_dw_small(const int32_t *stages, int E, int N, int K, int f32, int accumulate, int cus)
{
    int groups = 0, longest = 0, two = 0, four = 0;
    for (int e = 0; e < E; ++e) {
        if (accumulate && stages[e] == 0) continue;
        ++groups;
        longest = std::max(longest, stages[e]);
        two += std::max(stages[e], 2);
        four += std::max(stages[e], 4);
    }
    return dbs::moe_dw_small(groups, longest, two, four, N, K, f32, dbs::moe_dw_grid(E, N, K, cus));
}

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

constexpr int64_t kMaxRows = int64_t(1) << 25;      // rows of the sorted order
constexpr int64_t kMaxWidth = int64_t(1) << 21;     // N and K
constexpr int64_t kGatherLimit = 0xFF000000;        // bytes of a gathered X
constexpr int64_t kTwoGiB = int64_t(1) << 31;
constexpr int64_t kMostTiles = int64_t(1) << 30;

// What gemm_moe_bf16, gemm_moe_swiglu_bf16 and gemm_moe_dw_bf16 share.
dbs_status check_product(const void *X, const void *other, const void *out, const int32_t *offsets,
                         const int32_t *rows, int64_t T, int64_t M, int64_t E, int64_t N, int64_t K)
{
    if (!X || !other || !out || !offsets) return fail(DBS_EINVAL, "null pointer argument");
    if (T <= 0 || M <= 0 || E <= 0 || N <= 0 || K <= 0) return fail(DBS_EINVAL, "T, M, E, N and K must be positive");
    if (T > kMaxRows || M > kMaxRows) return fail(DBS_EINVAL, "T or M above 2^25");
    if (E > dbs::kMoeMaxExperts) return fail(DBS_EINVAL, "more than 1024 experts");
    if (N > kMaxWidth || K > kMaxWidth) return fail(DBS_EINVAL, "N or K above 2^21");
    if (K % 8) return fail(DBS_EINVAL, "K must be a multiple of 8");
    if (!rows && T != M) return fail(DBS_EINVAL, "without row indices X must have M rows");
    if (!aligned(X, 16) || !aligned(other, 16)) return fail(DBS_EINVAL, "operands must be 16-byte aligned");
    if (!aligned(out, 2)) return fail(DBS_EINVAL, "the output must be 2-byte aligned");
    if (!aligned(offsets, 4) || (rows && !aligned(rows, 4)))
        return fail(DBS_EINVAL, "offsets and rows must be 4-byte aligned");
    if (N * K * 2 >= kTwoGiB) return fail(DBS_EUNSUPPORTED, "an expert's matrix of 2 GiB or more");
    if (rows && T * K * 2 > kGatherLimit) return fail(DBS_EUNSUPPORTED, "a gathered X of nearly 4 GiB or more");
    return DBS_OK;
}

dbs_status run_product(dbs::MoeGemm p, hipStream_t stream)
{
    // the kernels number their tiles (64 x 32 the smallest) in int, with a round of workgroups to spare
    if (((int64_t)p.M / 64 + p.E) * (((int64_t)p.ncols + 31) / 32) >= kMostTiles)
        return fail(DBS_EUNSUPPORTED, "too many output tiles");
    int cus = 0;
    const int st = dbs::device_compute_units(&cus);
    if (st != DBS_OK) return (dbs_status)st;
    p.vec = p.ncols % 8 == 0 && aligned(p.D, 16);
    const int height = dbs::moe_tile_rows(p.M, p.E, p.N, p.ncols, p.wmn, p.gate, cus);
    return done(dbs::launch_moe_tiles(p, height, cus, stream));
}

dbs::MoeGemm product(const void *X, const void *W, void *D, const int32_t *offsets, const int32_t *rows, int64_t T,
                     int64_t M, int64_t E, int64_t N, int64_t K)
{
    dbs::MoeGemm p{};
    p.X = static_cast<const uint8_t *>(X);
    p.W = static_cast<const uint8_t *>(W);
    p.D = static_cast<uint8_t *>(D);
    p.offsets = offsets;
    p.rows = rows;
    p.T = T;
    p.M = (int)M;
    p.E = (int)E;
    p.N = (int)N;
    p.K = (int)K;
    p.ncols = (int)N;
    return p;
}

dbs_status check_route(dbs_real type, const void *logits, int64_t T, int64_t E, int64_t k)
{
    if (!logits) return fail(DBS_EINVAL, "null pointer argument");
    if (type != DBS_F32 && type != DBS_BF16) return fail(DBS_EINVAL, "unknown logit type");
    if (T <= 0 || E <= 0 || k <= 0) return fail(DBS_EINVAL, "T, E and k must be positive");
    if (E > dbs::kMoeMaxExperts) return fail(DBS_EINVAL, "more than 1024 experts");
    if (k > E) return fail(DBS_EINVAL, "k above the number of experts");
    if (k > dbs::kMoeMaxK) return fail(DBS_EUNSUPPORTED, "more than 16 experts per token");
    if (T > kMaxRows / k) return fail(DBS_EINVAL, "T * k above 2^25");
    if (!aligned(logits, type == DBS_F32 ? 4 : 2)) return fail(DBS_EINVAL, "misaligned logits");
    return DBS_OK;
}

dbs_status check_route_outputs(const int32_t *experts, const float *weights, const int32_t *offsets,
                               const int32_t *rows, const int32_t *slots, const void *workspace, size_t workspace_bytes,
                               int64_t need, uintptr_t alignment)
{
    if (!experts || !weights || !offsets || !rows || !slots) return fail(DBS_EINVAL, "null pointer argument");
    if (!aligned(experts, 4) || !aligned(weights, 4) || !aligned(offsets, 4) || !aligned(rows, 4) || !aligned(slots, 4))
        return fail(DBS_EINVAL, "misaligned output");
    if (need > 0 && (!workspace || !aligned(workspace, alignment) || workspace_bytes < (size_t)need))
        return fail(DBS_EINVAL, "workspace missing, misaligned or too small");
    return DBS_OK;
}

dbs_status check_score(dbs_score score, int renormalize, float scale)
{
    if (score != DBS_SOFTMAX && score != DBS_SIGMOID) return fail(DBS_EINVAL, "unknown score");
    if (renormalize != 0 && renormalize != 1) return fail(DBS_EINVAL, "renormalize must be 0 or 1");
    if (!std::isfinite(scale)) return fail(DBS_EINVAL, "scale must be finite");
    return DBS_OK;
}

dbs_status check_rows(int64_t rows, int64_t width)
{
    if (rows <= 0 || width <= 0) return fail(DBS_EINVAL, "sizes must be positive");
    if (rows > kMaxRows || width > kMaxWidth) return fail(DBS_EINVAL, "rows above 2^25 or width above 2^21");
    return DBS_OK;
}

}  // namespace

extern "C" {

size_t moe_route_workspace(int64_t T, int64_t E, int64_t k)
{
    if (T <= 0 || E <= 0 || k <= 0 || E > dbs::kMoeMaxExperts || k > E || k > dbs::kMoeMaxK || T > kMaxRows / k) return 0;
    return (size_t)dbs::moe_route_workspace_bytes(T, E);
}

dbs_status moe_route(dbs_real type, const void *logits, int64_t T, int64_t E, int64_t k, int renormalize,
                     int32_t *experts, float *weights, int32_t *offsets, int32_t *rows, int32_t *slots,
                     void *workspace, size_t workspace_bytes, hipStream_t stream)
{
    dbs_status st = check_route(type, logits, T, E, k);
    if (st != DBS_OK) return st;
    if (renormalize != 0 && renormalize != 1) return fail(DBS_EINVAL, "renormalize must be 0 or 1");
    if ((st = check_route_outputs(experts, weights, offsets, rows, slots, workspace, workspace_bytes,
                                  dbs::moe_route_workspace_bytes(T, E), 4)) != DBS_OK)
        return st;
    dbs::MoeRoute p{logits, type == DBS_BF16, T, (int)E, (int)k, renormalize, experts, weights, offsets, rows, slots,
                    static_cast<int32_t *>(workspace)};
    return done(dbs::launch_moe_route(p, stream));
}

dbs_status moe_route_bwd(dbs_real type, const void *logits, int64_t T, int64_t E, int64_t k, int renormalize,
                         const int32_t *experts, const float *dweights, void *dlogits, hipStream_t stream)
{
    dbs_status st = check_route(type, logits, T, E, k);
    if (st != DBS_OK) return st;
    if (!experts || !dweights || !dlogits) return fail(DBS_EINVAL, "null pointer argument");
    if (!aligned(experts, 4) || !aligned(dweights, 4) || !aligned(dlogits, type == DBS_F32 ? 4 : 2))
        return fail(DBS_EINVAL, "misaligned array");
    if (renormalize != 0 && renormalize != 1) return fail(DBS_EINVAL, "renormalize must be 0 or 1");
    return done(dbs::launch_moe_route_bwd(logits, type == DBS_BF16, T, (int)E, (int)k, 0, renormalize, 1.0f, experts, dweights,
                                          dlogits, stream));
}

size_t moe_route_grouped_workspace(int64_t T, int64_t E, int64_t k)
{
    if (T <= 0 || E <= 0 || k <= 0 || E > dbs::kMoeMaxExperts || k > E || k > dbs::kMoeMaxK || T > kMaxRows / k) return 0;
    return (size_t)dbs::moe_route_grouped_workspace_bytes(T, E);
}

dbs_status moe_route_grouped(dbs_real type, const void *logits, const float *bias, int64_t T, int64_t E, int64_t k,
                             dbs_score score, int64_t groups, int64_t kept_groups, int64_t group_best, int renormalize,
                             float scale, int32_t *experts, float *weights, int32_t *offsets, int32_t *rows,
                             int32_t *slots, void *workspace, size_t workspace_bytes, hipStream_t stream)
{
    dbs_status st = check_route(type, logits, T, E, k);
    if (st != DBS_OK) return st;
    if ((st = check_score(score, renormalize, scale)) != DBS_OK) return st;
    if (groups <= 0 || groups > E || E % groups) return fail(DBS_EINVAL, "groups must divide the number of experts");
    if (kept_groups <= 0 || kept_groups > groups) return fail(DBS_EINVAL, "kept_groups outside 1 .. groups");
    if (group_best != 1 && group_best != 2) return fail(DBS_EINVAL, "group_best must be 1 or 2");
    if (k > kept_groups * (E / groups)) return fail(DBS_EINVAL, "k above the number of experts in the kept groups");
    if (groups > dbs::kMoeMaxGroups) return fail(DBS_EUNSUPPORTED, "more than 16 groups");
    if (dbs::moe_route_grouped_lane(E, groups, true) > dbs::kMoeLaneExperts)
        return fail(DBS_EUNSUPPORTED, "groups too large: more than 64 experts of one to a lane");
    if ((st = check_route_outputs(experts, weights, offsets, rows, slots, workspace, workspace_bytes,
                                  dbs::moe_route_grouped_workspace_bytes(T, E), 16)) != DBS_OK)
        return st;
    if (!aligned(bias, 4)) return fail(DBS_EINVAL, "misaligned bias");
    dbs::MoeRouteGrouped g{};
    g.r = dbs::MoeRoute{logits, type == DBS_BF16, T, (int)E, (int)k, renormalize, experts, weights, offsets, rows, slots,
                        static_cast<int32_t *>(workspace)};
    g.bias = bias;
    g.sigmoid = score == DBS_SIGMOID;
    g.groups = (int)groups;
    g.kept = (int)kept_groups;
    g.best = (int)group_best;
    g.scale = scale;
    return done(dbs::launch_moe_route_grouped(g, stream));
}

dbs_status moe_route_grouped_bwd(dbs_real type, const void *logits, int64_t T, int64_t E, int64_t k, dbs_score score,
                                 int renormalize, float scale, const int32_t *experts, const float *dweights,
                                 void *dlogits, hipStream_t stream)
{
    dbs_status st = check_route(type, logits, T, E, k);
    if (st != DBS_OK) return st;
    if ((st = check_score(score, renormalize, scale)) != DBS_OK) return st;
    if (!experts || !dweights || !dlogits) return fail(DBS_EINVAL, "null pointer argument");
    if (!aligned(experts, 4) || !aligned(dweights, 4) || !aligned(dlogits, type == DBS_F32 ? 4 : 2))
        return fail(DBS_EINVAL, "misaligned array");
    return done(dbs::launch_moe_route_bwd(logits, type == DBS_BF16, T, (int)E, (int)k, score == DBS_SIGMOID, renormalize,
                                          scale, experts, dweights, dlogits, stream));
}

dbs_status gemm_moe_bf16(const void *X, const void *W, void *D, const int32_t *offsets, const int32_t *rows,
                         int64_t T, int64_t M, int64_t E, int64_t N, int64_t K, dbs_layout lw, hipStream_t stream)
{
    dbs_status st = check_product(X, W, D, offsets, rows, T, M, E, N, K);
    if (st != DBS_OK) return st;
    if (lw != DBS_K_MAJOR && lw != DBS_MN_MAJOR) return fail(DBS_EINVAL, "unknown layout value");
    if (lw == DBS_MN_MAJOR && N % 8)
        return fail(DBS_EUNSUPPORTED, "MN-major W needs N to be a multiple of 8 (16-byte rows)");
    dbs::MoeGemm p = product(X, W, D, offsets, rows, T, M, E, N, K);
    p.wmn = lw == DBS_MN_MAJOR;
    return run_product(p, stream);
}

dbs_status gemm_moe_swiglu_bf16(const void *X, const void *W, void *D, const int32_t *offsets, const int32_t *rows,
                                int64_t T, int64_t M, int64_t E, int64_t F, int64_t K, hipStream_t stream)
{
    if (F > kMaxWidth / 2) return fail(DBS_EINVAL, "F above 2^20");
    dbs_status st = check_product(X, W, D, offsets, rows, T, M, E, 2 * F, K);
    if (st != DBS_OK) return st;
    dbs::MoeGemm p = product(X, W, D, offsets, rows, T, M, E, 2 * F, K);
    p.ncols = (int)F;
    p.gate = 1;
    return run_product(p, stream);
}

dbs_status gemm_moe_dw_bf16(dbs_real type, const void *dY, const void *X, void *dW, const int32_t *offsets,
                            const int32_t *rows, int64_t T, int64_t M, int64_t E, int64_t N, int64_t K,
                            int accumulate, hipStream_t stream)
{
    dbs_status st = check_product(X, dY, dW, offsets, rows, T, M, E, N, K);
    if (st != DBS_OK) return st;
    if (N % 8) return fail(DBS_EINVAL, "N must be a multiple of 8");
    if (type != DBS_F32 && type != DBS_BF16) return fail(DBS_EINVAL, "unknown output type");
    if (accumulate != 0 && accumulate != 1) return fail(DBS_EINVAL, "accumulate must be 0 or 1");
    if (accumulate && type != DBS_F32) return fail(DBS_EUNSUPPORTED, "accumulation needs an fp32 dW");
    if (!aligned(dW, 16)) return fail(DBS_EINVAL, "dW must be 16-byte aligned");
    // (the kernel numbers its tiles, 64 x 128 the smaller ones, in int: N K < 2^30 and widths up to 2^21
    // make fewer than 2^17 + 2^15 + 2^14 + 2 of an expert, 2^28 over 1024 experts)
    int cus = 0;
    const int e = dbs::device_compute_units(&cus);
    if (e != DBS_OK) return (dbs_status)e;
    dbs::MoeGemmDw p{static_cast<const uint8_t *>(dY), static_cast<const uint8_t *>(X), static_cast<uint8_t *>(dW),
                     offsets, rows, T, (int)M, (int)E, (int)N, (int)K, type == DBS_F32, accumulate};
    return done(dbs::launch_moe_dw(p, cus, stream));
}

dbs_status swiglu_bf16(const void *H, void *A, int64_t M, int64_t F, hipStream_t stream)
{
    if (!H || !A) return fail(DBS_EINVAL, "null pointer argument");
    dbs_status st = check_rows(M, F);
    if (st != DBS_OK) return st;
    if (!aligned(H, 2) || !aligned(A, 2)) return fail(DBS_EINVAL, "arrays must be 2-byte aligned");
    return done(dbs::launch_swiglu(H, A, M, F, stream));
}

dbs_status swiglu_bwd_bf16(const void *dA, const void *H, void *dH, int64_t M, int64_t F, hipStream_t stream)
{
    if (!dA || !H || !dH) return fail(DBS_EINVAL, "null pointer argument");
    dbs_status st = check_rows(M, F);
    if (st != DBS_OK) return st;
    if (!aligned(H, 2) || !aligned(dA, 2) || !aligned(dH, 2)) return fail(DBS_EINVAL, "arrays must be 2-byte aligned");
    return done(dbs::launch_swiglu_bwd(dA, H, dH, M, F, stream));
}

static dbs_status check_combine(int64_t T, int64_t M, int64_t k, int64_t H)
{
    if (T <= 0 || k <= 0) return fail(DBS_EINVAL, "sizes must be positive");
    if (k > dbs::kMoeMaxK) return fail(DBS_EUNSUPPORTED, "more than 16 experts per token");
    if (T > kMaxRows || T * k > kMaxRows) return fail(DBS_EINVAL, "T * k above 2^25");
    return check_rows(M, H);
}

dbs_status moe_combine_bf16(const void *Y, const int32_t *slots, const float *weights, void *out, int64_t T,
                            int64_t M, int64_t k, int64_t H, hipStream_t stream)
{
    if (!Y || !slots || !out) return fail(DBS_EINVAL, "null pointer argument");
    dbs_status st = check_combine(T, M, k, H);
    if (st != DBS_OK) return st;
    if (!aligned(Y, 2) || !aligned(out, 2) || !aligned(slots, 4) || !aligned(weights, 4))
        return fail(DBS_EINVAL, "misaligned array");
    return done(dbs::launch_moe_combine(Y, slots, weights, out, T, M, (int)k, H, stream));
}

dbs_status moe_combine_bwd_bf16(const void *dO, const void *Y, const int32_t *slots, const float *weights,
                                const int32_t *offsets, int64_t E, void *dY, float *dweights, int64_t T, int64_t k,
                                int64_t H, hipStream_t stream)
{
    if (!dO || !Y || !slots || !weights || !offsets || !dY || !dweights)
        return fail(DBS_EINVAL, "null pointer argument");
    dbs_status st = check_combine(T, T * k, k, H);
    if (st != DBS_OK) return st;
    if (E <= 0 || E > dbs::kMoeMaxExperts) return fail(DBS_EINVAL, "E outside 1 .. 1024");
    if (!aligned(dO, 2) || !aligned(Y, 2) || !aligned(dY, 2) || !aligned(slots, 4) || !aligned(weights, 4) ||
        !aligned(offsets, 4) || !aligned(dweights, 4))
        return fail(DBS_EINVAL, "misaligned array");
    return done(dbs::launch_moe_combine_bwd(dO, Y, slots, weights, offsets + E, dY, dweights, T, T * k, (int)k, H,
                                            stream));
}

}  // extern "C"
