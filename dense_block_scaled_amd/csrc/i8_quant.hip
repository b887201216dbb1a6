// i8_quant.hip -- gfx950 kernel of the row quantiser:
//
//     scale[m] = amax_m / 127,  codes[m, k] = the whole number nearest to 127 x[m, k] / amax_m     amax_m = max_k |x[m, k]|
//
// Ties go to the even number, and the choice is that of the exact quotient:
// t = x (127 / amax) in fp32 is within 127 2^-23 < 2^-16 of it, so a t further
// than 2^-15 from a tie m + 1/2 has its neighbour; nearer, the
// products 254 |x| and (2 m + 1) amax decide, 32 bits each and exact in fp64.
// A row of zeros has scale 0; one with an infinity or a NaN has
// scale NaN and codes 0, so that every product with it is NaN.
//
// One pass: a row's pieces stay in registers between the maximum and the codes
// (rows longer than LANES x 8 x P elements read the rest again).  Memory bounds it: 32768
// rows of 4096 bf16 take 65 us, 6.2 TB/s read and written (a copy has 5.1 TB/s); 48 such
// rows 3.4 us, the way into the kernel and two trips to memory.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "i8.h"

namespace dbs {
namespace {

typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;
typedef __attribute__((ext_vector_type(2))) uint32_t u32x2;
constexpr int kThreads = 256;

// V elements as they lie in memory (8, or 1 where rows are not whole pieces)
template <bool BF16, int V>
struct Raw {
    static constexpr int kWords = V == 1 ? 1 : BF16 ? 4 : 8;
    uint32_t w[kWords];

    __device__ __forceinline__ void load(const void *x, int64_t at)
    {
        if constexpr (V == 1) {
            w[0] = BF16 ? (uint32_t) reinterpret_cast<const uint16_t *>(x)[at] << 16 : reinterpret_cast<const uint32_t *>(x)[at];
        } else {
            const u32x4 *q = reinterpret_cast<const u32x4 *>(reinterpret_cast<const uint8_t *>(x) + at * (BF16 ? 2 : 4));
#pragma unroll
            for (int i = 0; i < kWords / 4; ++i) {
                const u32x4 v = __builtin_nontemporal_load(q + i);
#pragma unroll
                for (int j = 0; j < 4; ++j) w[4 * i + j] = v[j];
            }
        }
    }
    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0;
    }
    __device__ __forceinline__ uint32_t bits(int i) const      // of element i as fp32
    {
        if constexpr (V == 1 || !BF16) return w[i];
        else return i & 1 ? w[i >> 1] & 0xFFFF0000u : w[i >> 1] << 16;
    }
};

struct Row {
    float amax, inv, pre;     // pre: 1, or what brings a tiny row to where 127 / amax is finite
};

__device__ __forceinline__ int code(uint32_t bits, const Row &r)
{
    const float x = __builtin_bit_cast(float, bits) * r.pre, t = x * r.inv, n = __builtin_rintf(t);
    int c = (int)n;
    if (__builtin_expect(fabsf(fabsf(t - n) - 0.5f) < 0x1p-15f, 0)) {
        const float m = floorf(fabsf(t));
        const double q = 254.0 * (double)fabsf(x), mid = (double)(2.0f * m + 1.0f) * (double)r.amax;
        const int up = q > mid || (q == mid && ((int)m & 1));
        c = (int)m + up;
        c = x < 0.0f ? -c : c;
    }
    return c;
}

// LANES threads a row (64: four rows a workgroup, each a wave's own; 256: one).
template <bool BF16, int V, int LANES, int P>
__global__ __launch_bounds__(kThreads) void quant_i8_kernel(const void *x, int64_t M, int64_t K, int8_t *codes, float *scales)
{
    static_assert(LANES == 64 || LANES == kThreads, "a wave or a workgroup a row");
    __shared__ uint32_t part[kThreads / 64];
    const int l = threadIdx.x % LANES;
    const int64_t m = (int64_t)blockIdx.x * (kThreads / LANES) + threadIdx.x / LANES;
    if (m >= M) return;                          // (uniform in the threads of a row)
    const int64_t at = m * K, pieces = K / V;
    Raw<BF16, V> v[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
        if (i * LANES + l < pieces) v[i].load(x, at + (int64_t)(i * LANES + l) * V);
        else v[i].zero();
    }
    uint32_t most = 0;                           // fp32 magnitudes order as their bits; a NaN's are the largest
    auto larger = [&](const Raw<BF16, V> &r) {
#pragma unroll
        for (int q = 0; q < V; ++q) most = max(most, r.bits(q) & 0x7FFFFFFFu);
    };
#pragma unroll
    for (int i = 0; i < P; ++i) larger(v[i]);
    for (int64_t i = P * LANES + l; i < pieces; i += LANES) {
        Raw<BF16, V> r;
        r.load(x, at + i * V);
        larger(r);
    }
#pragma unroll
    for (int d = 32; d; d /= 2) most = max(most, (uint32_t)__shfl_xor((int)most, d));
    if constexpr (LANES == kThreads) {
        if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = most;
        __syncthreads();
        most = max(max(part[0], part[1]), max(part[2], part[3]));
    }
    const bool good = most < 0x7F800000u && most > 0;
    Row r;
    r.amax = __builtin_bit_cast(float, most);
    if (l == 0) scales[m] = most < 0x7F800000u ? r.amax / 127.0f : __builtin_nanf("");
    r.pre = r.amax < 0x1p-100f ? 0x1p64f : 1.0f;
    r.amax *= r.pre;
    r.inv = good ? 127.0f / r.amax : 0.0f;
    auto write = [&](const Raw<BF16, V> &raw, int64_t i) {
        int c[V];
#pragma unroll
        for (int q = 0; q < V; ++q) c[q] = good ? code(raw.bits(q), r) : 0;
        int8_t *to = codes + at + i * V;
        if constexpr (V == 1) {
            *to = (int8_t)c[0];
        } else {
            u32x2 w;
#pragma unroll
            for (int h = 0; h < 2; ++h)
                w[h] = (c[4 * h] & 0xFF) | (c[4 * h + 1] & 0xFF) << 8 | (c[4 * h + 2] & 0xFF) << 16 | (uint32_t)c[4 * h + 3] << 24;
            *reinterpret_cast<u32x2 *>(to) = w;
        }
    };
#pragma unroll
    for (int i = 0; i < P; ++i)
        if (i * LANES + l < pieces) write(v[i], i * LANES + l);
    for (int64_t i = P * LANES + l; i < pieces; i += LANES) {
        Raw<BF16, V> raw;
        raw.load(x, at + i * V);
        write(raw, i);
    }
}

// Rows of a launch: HIP takes grids of fewer than 2^32 threads, and a row has up to kThreads of them
constexpr int64_t kLaunchRows = int64_t(1) << 23;

hipError_t launch_rows(const void *x, int bf16, int64_t M, int64_t K, int8_t *codes, float *scales, hipStream_t stream)
{
    auto go = [&](auto b, auto v, auto lanes, auto p) {
        constexpr int L = decltype(lanes)::value;
        const dim3 grid((uint32_t)((M + kThreads / L - 1) / (kThreads / L)));
        hipLaunchKernelGGL((quant_i8_kernel<decltype(b)::value, decltype(v)::value, L, decltype(p)::value>), grid,
                           dim3(kThreads), 0, stream, x, M, K, codes, scales);
        return hipGetLastError();
    };
    using W = std::integral_constant<int, 64>;
    using G = std::integral_constant<int, kThreads>;
    using I1 = std::integral_constant<int, 1>;
    using I2 = std::integral_constant<int, 2>;
    using I4 = std::integral_constant<int, 4>;
    using I8 = std::integral_constant<int, 8>;
    auto by_size = [&](auto b) {
        const bool whole = K % 8 == 0 && ((reinterpret_cast<uintptr_t>(x) & 15) | (reinterpret_cast<uintptr_t>(codes) & 7)) == 0;
        if (!whole) return go(b, I1{}, G{}, I8{});
        // A workgroup a row has the row's pieces under way in one trip, a wave a row none of the
        // waiting for the others: us of rows x K, wave / workgroup, bf16 then fp32:
        //     48 x 1024    3.9 /  3.3    3.5 /  3.2        48 x 2048    4.7 /  3.3    4.4 /  3.2
        //   4096 x 1024    5.7 /  6.7    6.5 /  6.9      8192 x 2048     15 /   14     19 /   17
        //  32768 x 1024     21 /   36     31 /   35     32768 x 2048     38 /   46     60 /   57
        //  32768 x  512     15 /   29     17 /   30     32768 x 4096     78 /   68    117 /  114
        constexpr bool BF16 = decltype(b)::value;
        if (K <= 64 * 8) return go(b, I8{}, W{}, I1{});
        if (K <= 64 * 8 * 2 && M >= 4096) return go(b, I8{}, W{}, I2{});
        if constexpr (BF16) {
            if (K <= 64 * 8 * 4 && M >= 16384) return go(b, I8{}, W{}, I4{});
        }
        if (K <= 256 * 8) return go(b, I8{}, G{}, I1{});
        if (K <= 256 * 8 * 2) return go(b, I8{}, G{}, I2{});
        if (K <= 256 * 8 * 4) return go(b, I8{}, G{}, I4{});
        return go(b, I8{}, G{}, I8{});
    };
    return bf16 ? by_size(std::true_type{}) : by_size(std::false_type{});
}

}  // namespace

hipError_t launch_quant_i8(const void *x, int bf16, int64_t M, int64_t K, int8_t *codes, float *scales, hipStream_t stream)
{
    for (int64_t m = 0; m < M; m += kLaunchRows) {
        const hipError_t e = launch_rows(static_cast<const uint8_t *>(x) + m * K * (bf16 ? 2 : 4), bf16,
                                         M - m < kLaunchRows ? M - m : kLaunchRows, K, codes + m * K, scales + m, stream);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace dbs
