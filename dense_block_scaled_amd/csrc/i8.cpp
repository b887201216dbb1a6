// i8.cpp -- the C ABI of the 8-bit integer operators declared in include/dbs.h:
// argument validation, choice of kernel and launch.
#include "i8.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdio>

#include "dbs.h"
#include "launch.h"
#include "moe.h"

namespace dbs {

// The tile with the least estimated time, in us: a first round of tiles over the
// CUs (the walk along K, `k` times 1024 long, behind the way into the kernel and
// out of it), further rounds at what a busy machine takes, or the reading of W at
// 5.5 TB/s where that is more.  Groups (E > 1) are known on the device only: M / E rows of
// each, half a tile of each is waste, some may have none; tiles then even out,
// and rounds are counted in parts.  (D's and X's bytes are not in it: 1075 x 28672 x 1024,
// 62 MB of results, gets 128 x 128 tiles at 55 us where 256 x 256 take 45.)  us of the dense product, W from memory, with tiles of
//
//                        16 x 16  16 x 64  64 x 16  64 x 32  64 x 64  128 x 64  128 x 128  256 x 256
//      1 x 4096 x 4096       5.8      9.3      9.0      9.6       11        14         19         36
//     16 x 8192 x 4096        12       10       14       10       12        15         19         36
//     48 x 4096 x 4096        18       11      9.5       11       13        15         20         36
//    128 x 8192 x 4096        63       39       24       18       14        18         23         40
//    128 x 11008 x 8192      169      110       62       45       41        32         43         72
//    512 x 4096 x 4096       121       75       41       29       21        18         23         46
//    512 x 8192 x 1024       111       43       40       24       15        13         11         19
//   1024 x 4096 x 4096       237      146       75       51       35        30         24         48
//   2048 x 4096 x 4096       477      289      142       95       64        55         42         52
//   4096 x 4096 x 4096       956      581      274      182      123       104         78         59
//
// of 1 / 4 / 16 / 48 tokens each to 8 of 64 experts of 2048 x 1408 with 16 x 64 8.7 / 17.0 / 26.4 / 34.6,
// with 64 x 64 9.4 / 18.6 / 29.5 / 38.2, and of 16 .. 8191 tokens each to 4 of 32 experts of 2056 x 4096 with
// 64 x 64 / 128 x 128 / 256 x 256 47 / 47 / 45 for 16 tokens (16 x 64: 44), 75 / 69 / 79 for 512, 102 / 94 / 86 for 1024,
// 559 / 369 / 281 for 8191.  Over 80 dense sizes drawn at random the tile chosen takes 0.9 % longer than the fastest
// (22 % at most), over 60 sizes of experts 2.6 % (23 %).
I8Tile i8_tile(int64_t M, int64_t E, int64_t N, int64_t ncols, int64_t K, bool gate, int cus, double *us)
{
    const double k = K / 1024.0, n = cus;
    const int64_t likely = (2 * M * E + 2 * M + E - 1) / (2 * M + E), met = E == 1 ? 1 : std::min(M, likely);
    auto tiles = [&](int64_t tm, int64_t tn) {
        const int64_t rows = E == 1 ? (M + tm - 1) / tm : std::max(M / tm + met / 2, met);
        const int64_t wide = gate ? tn / 2 : tn;
        return double(rows * ((ncols + wide - 1) / wide));
    };
    auto more = [&](double x) { return E == 1 ? std::max(std::ceil(x) - 1, 0.0) : std::max(x - 1, 0.0); };
    const double w = 4 + double(met) * N * K / 5.5e6;
    I8Tile best{64, 64};
    double least = 1e30;
    auto offer = [&](int rows, int cols, double t) {
        const double score = std::max(t, w) + 0.2 * t;
        if (score >= least) return;
        least = score;
        best = I8Tile{rows, cols};
        if (us) *us = std::max(t, w);
    };
    {
        // (not for more than the two tiles that a CU works on together)
        const double x = tiles(16, gate ? 32 : 16) / n, m = std::min(double(M) / met, 16.0) / 16, c = gate ? 1.6 : 1.0;
        if (x <= 2) offer(16, 16, 3.6 + c * k * (x <= 1 ? 0.36 + 0.37 * m : 0.95 + 0.7 * m));
    }
    auto deep = [&](int rows, int cols, double first, double next) {
        const double x = tiles(rows, cols) / n;
        offer(rows, cols, 4.8 + first * k + more(x) * (1.9 + next * k));
    };
    if (!gate) deep(64, 16, 0.6, 0.75);
    deep(64, 32, 0.95, 1.05);
    deep(64, 64, 1.42, 1.55);
    if (M <= 16 * met) deep(16, 64, 0.92, 1.0);    // (more rows read W again: 48 x 4096 x 4096 in 10.6 us)
    double x = tiles(128, 64) / n;
    // (of groups, whose rows are not known, 128 x 128 or 64 x 64 tiles were as fast or up to 20 % faster)
    if (E == 1 && !gate) offer(128, 64, 5.7 + (1.9 + 0.6 * std::min(x, 1.0)) * k + more(x) * (1.3 + 2.47 * k));
    x = tiles(128, 128) / n;
    offer(128, 128, 6.1 + (2.7 + 1.6 * std::min(x, 1.0)) * k + more(x) * (1.3 + 4.35 * k));
    x = tiles(256, 256) / n;
    offer(256, 256, 10 + (8.6 + 3.1 * std::min(x, 1.0)) * k + more(x) * (7 + 12.2 * k));
    return best;
}

// Tiles that fill the CUs a whole number of times and one more cost a round for
// the one.  The rows (or columns) of the whole rounds then go by themselves and
// the others behind them, where that saves more than 8 % and 2 us by the same
// estimate: 4539 x 4096 x 4096 in 75 us, not 95, 4688 x 4096 x 8192 in 138, not 182, 1302 x 12205 x 3296
// in 62, not 84, 992 x 4108 x 2320 in 22, not 28; with estimates nearer than that the two were up
// to 5 % slower (2280 x 12836 x 4480: 129 us, not 123).
I8Part i8_part(int64_t M, int64_t N, int64_t K, int cus)
{
    I8Part best{M, N};
    double whole = 0;
    i8_tile(M, 1, N, N, K, false, cus, &whole);
    if (whole < 20) return best;            // (nothing to save, and the trial takes the host 0.9 us)
    double least = whole / 1.08 - 2;
    auto offer = [&](int64_t rows, int64_t cols) {
        double a = 0, b = 0;
        if (rows <= 0 || cols <= 0 || (rows >= M && cols >= N)) return;
        i8_tile(rows, 1, cols, cols, K, false, cus, &a);
        const int64_t m = rows < M ? M - rows : M, n = cols < N ? N - cols : N;
        i8_tile(m, 1, n, n, K, false, cus, &b);
        if (a + b >= least) return;
        least = a + b;
        best = I8Part{rows, cols};
    };
    for (int t : {128, 256}) {
        const int64_t down = (M + t - 1) / t, across = (N + t - 1) / t, rounds = down * across / cus;
        if (rounds == 0) continue;
        offer(std::min(rounds * cus / across * t, M), N);
        offer(M, std::min(rounds * cus / down * t, N));
    }
    return best;
}

}  // namespace dbs

extern "C" int64_t dbs_i8_part(int64_t M, int64_t N, int64_t K, int cus)
{
    const dbs::I8Part p = dbs::i8_part(M, N, K, cus);
    return p.cols < N ? -p.cols : p.rows;
}

extern "C" int dbs_i8_tile(int64_t M, int64_t E, int64_t N, int64_t K, int gate, int cus)
{
    const dbs::I8Tile t = dbs::i8_tile(M, E, N, gate ? N / 2 : N, K, gate, cus);
    return 1000 * t.rows + t.cols;
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
    p.ldd = (int)N;
    return p;
}

dbs_status run_product(dbs::I8Gemm p, hipStream_t stream)
{
    // the kernels number their tiles in int, with a round of workgroups to spare (smaller ones than 64 x 32 only
    // where there are few)
    if (((int64_t)p.M / 64 + p.E) * (((int64_t)p.ncols + 31) / 32) >= kMostTiles)
        return fail(DBS_EUNSUPPORTED, "too many output tiles");
    int cus = 0;
    const int st = dbs::device_compute_units(&cus);
    if (st != DBS_OK) return (dbs_status)st;
    p.vec = p.ldd % (p.f32 ? 4 : 8) == 0 && aligned(p.D, 16);
    auto launch = [&](const dbs::I8Gemm &q) {
        return dbs::launch_i8_tiles(q, dbs::i8_tile(q.M, q.E, q.N, q.ncols, q.K, q.gate, cus), cus, stream);
    };
    if (p.offsets) return done(launch(p));
    const dbs::I8Part part = dbs::i8_part(p.M, p.N, p.K, cus);
    dbs::I8Gemm first = p;
    first.M = (int)part.rows;
    first.T = part.rows;
    first.N = first.ncols = (int)part.cols;
    const hipError_t e = launch(first);
    if (e != hipSuccess || (part.rows == p.M && part.cols == p.N)) return done(e);
    // the other rows, or the other columns
    const int64_t m = part.rows < p.M ? part.rows : 0, n = part.cols < p.N ? part.cols : 0;
    p.X += m * p.K;
    p.sX += m;
    p.W += n * p.K;
    p.sW += n;
    p.D += (m * p.ldd + n) * (p.f32 ? 4 : 2);
    p.M -= (int)m;
    p.T -= m;
    p.N -= (int)n;
    p.ncols = p.N;
    return done(launch(p));
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
    p.ldd = (int)F;
    p.gate = 1;
    return run_product(p, stream);
}

}  // extern "C"
