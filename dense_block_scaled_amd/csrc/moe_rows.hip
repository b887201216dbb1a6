// moe_rows.hip -- gfx950 kernel of the experts' products for a few rows: the
// single token and the small decoding batch, where an expert's matrix is read
// for a handful of rows and the time is the reading.
//
//     D[i, n] = sum_k X[rows[i], k] W_g[n, k]          W_g K-major (N x K)
//     D[i, f] = silu(h[f]) h[F + f]                    with the gate
//
// Output tiles of 256 x 64 or 64 x 256 leave most CUs without work here (one
// token of 8 experts and 1408 gated columns: 88 tiles), so the work is cut
// finer and along K: a workgroup takes 32 rows of one expert's matrix (the 16
// gate and 16 up rows of 16 gated outputs) and its eight waves an eighth of K
// each, every wave with 16 loads of a KiB under way at once; the eight sums
// are added in LDS in a fixed order.  Rows go through
// v_mfma_f32_16x16x32_bf16 sixteen at a time; the fragments of W come
// straight from memory (nothing else reads them), those of X from the caches.
// A group of more than 16 rows reads its matrix again for every 16.
#include "gemm_kernel.h"
#include "moe.h"

namespace dbs {
namespace {

typedef __attribute__((ext_vector_type(4))) float f32x4;

constexpr int kWaves = 8;
constexpr uint32_t kRowOOB = 0xFF000000u;    // + a row's bytes (at most 2^22) still lies past every resource

// KW: waves along K; the other kWaves / KW take further rows of the matrix.
template <bool GATE, int KW>
__global__ __launch_bounds__(64 * kWaves) void moe_rows(MoeGemm p)
{
    constexpr int NB = 2, kSteps = 8;        // blocks of 16 rows of the matrix; k-steps of 32 under way
    constexpr int NBO = GATE ? NB / 2 : NB;  // blocks of 16 outputs
    __shared__ f32x4 part[kWaves][NB][64];
    constexpr int TNO = 16 * NBO;      // outputs per wave and row
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wk = w % KW, lda = p.K * 2, n0 = (blockIdx.x * (kWaves / KW) + w / KW) * TNO;

    // this workgroup's group: number blockIdx.y among those with rows; the
    // last row of all groups on the way
    const int begin = min(max(p.offsets[0], 0), p.M);
    int g = -1, lo = 0, hi = 0, seen = 0, end = begin;
    for (int g0 = 0; g0 < p.E; g0 += 64) {
        const int e = g0 + lane;
        // (clamped and made ascending, as the tile kernels read them)
        int b = e < p.E ? max(min(max(p.offsets[e + 1], 0), p.M), end) : end;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const int o = __shfl_up(b, d);
            if (lane >= d) b = max(b, o);
        }
        const int before = __shfl_up(b, 1), a = lane == 0 ? end : before;
        const uint64_t has = __ballot(e < p.E && b > a);
        const int want = (int)blockIdx.y - seen, n = __popcll(has);
        if (g < 0 && want < n) {
            uint64_t rest = has;
            for (int i = 0; i < want; ++i) rest &= rest - 1;
            const int src = __ffsll((unsigned long long)rest) - 1;
            g = g0 + src;
            lo = __shfl(a, src);
            hi = __shfl(b, src);
        }
        seen += n;
        end = __shfl(b, 63);
    }
    g = __builtin_amdgcn_readfirstlane(g);
    lo = __builtin_amdgcn_readfirstlane(lo);
    hi = __builtin_amdgcn_readfirstlane(hi);

    // rows before the first group and behind the last are zero
    auto zero = [&](int64_t from, int64_t to) {
        const int64_t all = (int64_t)gridDim.x * gridDim.y * blockDim.x;
        for (int64_t i = from + ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * blockDim.x + threadIdx.x; i < to; i += all)
            reinterpret_cast<uint16_t *>(p.D)[i] = 0;
    };
    zero(0, (int64_t)begin * p.ncols);
    zero((int64_t)end * p.ncols, (int64_t)p.M * p.ncols);
    if (g < 0) return;

    // The wave's share of K in whole lines of 64 elements.  Lane l holds row
    // l % 16 and K 8 (l / 16) .. of a k-step, for X and W alike.
    const int per = (p.K + KW * 64 - 1) / (KW * 64) * 64;
    const int k0 = min(wk * per, p.K), k1 = min(k0 + per, p.K);
    const int kl = 8 * (lane >> 4);
    const int64_t wbytes = (int64_t)p.N * p.K * 2, at = (int64_t)n0 * lda;
    const __amdgpu_buffer_rsrc_t rw = make_rsrc(p.W + g * wbytes + at, n0 < p.ncols ? (uint32_t)(wbytes - at) : 0u);
    const uint32_t wrow = (uint32_t)((lane & 15) * lda), up = (uint32_t)(p.ncols * (int64_t)lda);

    for (int r0 = lo; r0 < hi; r0 += 16) {
        const int r = r0 + (lane & 15);
        uint32_t xrow = kRowOOB;
        uint32_t have;
        const uint8_t *xbase;
        if (p.rows) {
            const uint32_t t = r < hi ? (uint32_t)p.rows[r] : ~0u;
            xrow = t < (uint32_t)p.T ? t * (uint32_t)lda : kRowOOB;
            xbase = p.X;
            have = (uint32_t)p.T * (uint32_t)lda;
        } else {
            xrow = r < hi ? (uint32_t)((lane & 15) * lda) : kRowOOB;
            xbase = p.X + (int64_t)r0 * lda;
            have = (uint32_t)min(hi - r0, 16) * (uint32_t)lda;
        }
        const __amdgpu_buffer_rsrc_t rx = make_rsrc(xbase, have);
        f32x4 acc[NB] = {};
        for (int k = k0; k < k1; k += 32 * kSteps) {
            i32x4 a[kSteps], b[kSteps][NB];
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                const int kk = k + 32 * s + kl;
                const bool in = kk < k1;
#pragma unroll
                for (int u = 0; u < NB; ++u)
                    b[s][u] = __builtin_amdgcn_raw_buffer_load_b128(rw, in ? wrow + (u % NBO) * 16 * lda + (u / NBO) * up + 2 * kk : kOOB, 0, 0);
                a[s] = __builtin_amdgcn_raw_buffer_load_b128(rx, in ? xrow + 2 * kk : kRowOOB, 0, 0);
            }
#pragma unroll
            for (int s = 0; s < kSteps; ++s)
#pragma unroll
                for (int u = 0; u < NB; ++u)
                    acc[u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, b[s][u]),
                                                                    __builtin_bit_cast(bf16x8, a[s]), acc[u], 0, 0, 0);
        }
        // lane l: row l % 16, W rows 4 (l / 16) .. + 3 of block u
#pragma unroll
        for (int u = 0; u < NB; ++u) part[w][u][lane] = acc[u];
        __syncthreads();
        // waves of one place along the matrix take its blocks in turn
        for (int u = wk; u < NBO; u += KW) {
            f32x4 s0{}, s1{};
#pragma unroll
            for (int i = 0; i < KW; ++i) {
                s0 += part[w - wk + i][u][lane];
                if constexpr (GATE) s1 += part[w - wk + i][NBO + u][lane];
            }
            const int n = n0 + 16 * u + 4 * (lane >> 4);
            if (r < hi) {
                uint16_t *d = reinterpret_cast<uint16_t *>(p.D) + (int64_t)r * p.ncols;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float v = s0[q];
                    if constexpr (GATE) v = v * __builtin_amdgcn_rcpf(1.0f + __expf(-v)) * s1[q];
                    if (n + q < p.ncols) d[n + q] = (uint16_t)pack_bf16(v, 0.0f);
                }
            }
        }
        __syncthreads();
    }
}

}  // namespace

hipError_t launch_moe_rows(const MoeGemm &p, hipStream_t stream)
{
    auto go = [&](auto gate, auto kw) {
        constexpr bool GATE = decltype(gate)::value;
        constexpr int KW = decltype(kw)::value;
        const int tno = (GATE ? 16 : 32) * (kWaves / KW);
        const dim3 grid((p.ncols + tno - 1) / tno, p.M < p.E ? p.M : p.E);
        hipLaunchKernelGGL((moe_rows<GATE, KW>), grid, dim3(64 * kWaves), 0, stream, p);
        return hipGetLastError();
    };
    // A wave's share of K is what its loads under way cover (256), or half of
    // it: with K 768, 8 experts of 4096 outputs, 8 / 4 / 2 waves along K took
    // 21 / 16 / 16 us, with K 2048 and 2 experts 10 / 13 / 21 us.
    auto by_k = [&](auto gate) {
        if (p.K > 1024) return go(gate, std::integral_constant<int, 8>{});
        if (p.K > 512) return go(gate, std::integral_constant<int, 4>{});
        return go(gate, std::integral_constant<int, 2>{});
    };
    return p.gate ? by_k(std::true_type{}) : by_k(std::false_type{});
}

}  // namespace dbs
