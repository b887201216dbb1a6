// moe_pointwise.hip -- gfx950 kernels around the experts' products: the gate
// between them and the sum of a token's rows behind them, each with its
// gradient.  All are streams bound by memory; arithmetic is fp32, rounded
// once to bf16 on the way out.
//
//     swiglu         a = silu(g) u                  h = (g | u), silu(g) = g s, s = 1 / (1 + e^-g)
//     swiglu_bwd     dg = da u s (1 + g (1 - s)),   du = da g s
//     combine        out_t = sum_j w_tj Y[slot_tj]  (slots of -1 add nothing)
//     combine_bwd    dY[slot_tj] = w_tj dO_t,       dw_tj = <dO_t, Y[slot_tj]>
//
// Measured, where a copy of 1 GiB reaches 5.0 TB/s: swiglu 32768 x 2048 69 us
// (5.8 TB/s, two bytes read for one written), swiglu_bwd 49999 x 1416 129 us (5.5),
// combine 8192 tokens x 8 rows x 4096 116 us (5.2), combine_bwd 8191 x 6 x 2056
// 87 us (4.9, as much written as read).
//
// Every kernel has a form of 16-byte pieces (8 elements; row lengths that are
// multiples of 8, base addresses on 16 bytes) and one of single elements.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <initializer_list>
#include <type_traits>

#include "moe.h"
#include "moe_device.h"

namespace dbs {
namespace {

constexpr int kThreads = 256;

// V bf16 values as they lie in memory
template <int V>
struct Piece {
    uint32_t w[V / 2];
};
template <>
struct Piece<1> {
    uint16_t w[1];
};

template <int V>
__device__ __forceinline__ void unpack(const Piece<V> &p, float (&f)[V])
{
    if constexpr (V == 1) {
        f[0] = __builtin_bit_cast(float, (uint32_t)p.w[0] << 16);
    } else {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            f[2 * i] = __builtin_bit_cast(float, p.w[i] << 16);
            f[2 * i + 1] = __builtin_bit_cast(float, p.w[i] & 0xFFFF0000u);
        }
    }
}

template <int V>
__device__ __forceinline__ Piece<V> pack(const float (&f)[V])
{
    typedef __attribute__((ext_vector_type(2))) float f32x2;
    typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;
    Piece<V> p;
    if constexpr (V == 1) {
        p.w[0] = __builtin_bit_cast(uint16_t, (__bf16)f[0]);
    } else {
#pragma unroll
        for (int i = 0; i < V / 2; ++i)
            p.w[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{f[2 * i], f[2 * i + 1]}), bf16x2));
    }
    return p;
}

// Element i (a multiple of V) of a bf16 array
template <int V>
__device__ __forceinline__ Piece<V> load(const uint16_t *x, int64_t i)
{
    if constexpr (V == 1) {
        return Piece<1>{{x[i]}};
    } else {
        typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;
        return __builtin_bit_cast(Piece<V>, *reinterpret_cast<const u32x4 *>(x + i));
    }
}

template <int V>
__device__ __forceinline__ void store(uint16_t *x, int64_t i, const Piece<V> &p)
{
    if constexpr (V == 1) {
        x[i] = p.w[0];
    } else {
        typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;
        *reinterpret_cast<u32x4 *>(x + i) = __builtin_bit_cast(u32x4, p);
    }
}

// One piece of V outputs a thread: piece c of row m.
template <int V>
__global__ __launch_bounds__(kThreads) void swiglu_kernel(const uint16_t *H, uint16_t *A, int64_t pieces, int64_t F)
{
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < pieces; i += (int64_t)gridDim.x * kThreads) {
        const int64_t per = F / V, m = i / per, c = (i - m * per) * V;
        float g[V], u[V], a[V];
        unpack<V>(load<V>(H, m * 2 * F + c), g);
        unpack<V>(load<V>(H, m * 2 * F + F + c), u);
#pragma unroll
        for (int q = 0; q < V; ++q) a[q] = gated(g[q], u[q]);
        store<V>(A, m * F + c, pack<V>(a));
    }
}

template <int V>
__global__ __launch_bounds__(kThreads) void swiglu_bwd_kernel(const uint16_t *dA, const uint16_t *H, uint16_t *dH,
                                                              int64_t pieces, int64_t F)
{
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < pieces; i += (int64_t)gridDim.x * kThreads) {
        const int64_t per = F / V, m = i / per, c = (i - m * per) * V;
        float g[V], u[V], d[V], dg[V], du[V];
        unpack<V>(load<V>(H, m * 2 * F + c), g);
        unpack<V>(load<V>(H, m * 2 * F + F + c), u);
        unpack<V>(load<V>(dA, m * F + c), d);
#pragma unroll
        for (int q = 0; q < V; ++q) {
            const Sigmoid s = sigmoid(g[q]);
            const float ds = d[q] * s.p * s.r;
            dg[q] = ds * (u[q] * s.p) * (1.0f + g[q] * s.rest);
            du[q] = ds * (g[q] * s.p);
        }
        store<V>(dH, m * 2 * F + c, pack<V>(dg));
        store<V>(dH, m * 2 * F + F + c, pack<V>(du));
    }
}

// A slot as the kernels use it: -1 for anything that is no row of Y
__device__ __forceinline__ int slot_of(const int32_t *slots, int64_t p, int64_t M)
{
    const int s = slots[p];
    return s >= 0 && s < M ? s : -1;
}

template <int V>
__global__ __launch_bounds__(kThreads) void combine_kernel(const uint16_t *Y, const int32_t *slots,
                                                           const float *weights, uint16_t *out, int64_t pieces,
                                                           int64_t M, int k, int64_t H)
{
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < pieces; i += (int64_t)gridDim.x * kThreads) {
        const int64_t per = H / V, t = i / per, c = (i - t * per) * V;
        float acc[V] = {};
        // four rows under way at a time; a pair without a row reads row 0 and adds zeros
        for (int j0 = 0; j0 < k; j0 += 4) {
            int s[4];
            float w[4];
            Piece<V> y[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[j] = j0 + j < k ? slot_of(slots, t * k + j0 + j, M) : -1;
                w[j] = j0 + j < k && weights ? weights[t * k + j0 + j] : 1.0f;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] = load<V>(Y, (int64_t)max(s[j], 0) * H + c);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float f[V];
                unpack<V>(y[j], f);
#pragma unroll
                for (int q = 0; q < V; ++q) acc[q] = s[j] >= 0 ? acc[q] + w[j] * f[q] : acc[q];
            }
        }
        store<V>(out, t * H + c, pack<V>(acc));
    }
}

// One wave per pair (t, j): its row's gradient and its weight's.  Rows at or
// past *total have no pair: the wave of pair q zeroes row q if it is one.
template <int V>
__global__ __launch_bounds__(kThreads) void combine_bwd_kernel(const uint16_t *dO, const uint16_t *Y,
                                                               const int32_t *slots, const float *weights,
                                                               const int32_t *total, uint16_t *dY, float *dweights,
                                                               int64_t pairs, int64_t M, int k, int64_t H)
{
    const int lane = threadIdx.x & 63;
    const int64_t step = (int64_t)gridDim.x * (kThreads / 64);
    for (int64_t q = (int64_t)blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6); q < pairs; q += step) {
        const int64_t t = q / k;
        const int s = slot_of(slots, q, M);
        const float w = weights[q];
        float dot = 0.0f;
        if (s >= 0) {
            for (int64_t c = (int64_t)lane * V; c < H; c += 64 * V) {
                float d[V], y[V], g[V];
                unpack<V>(load<V>(dO, t * H + c), d);
                unpack<V>(load<V>(Y, (int64_t)s * H + c), y);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    dot += d[e] * y[e];
                    g[e] = w * d[e];
                }
                store<V>(dY, (int64_t)s * H + c, pack<V>(g));
            }
#pragma unroll
            for (int d = 32; d; d /= 2) dot += __shfl_xor(dot, d);
        }
        if (lane == 0) dweights[q] = dot;
        if (q >= *total)
            for (int64_t c = (int64_t)lane * V; c < H; c += 64 * V) store<V>(dY, q * H + c, Piece<V>{});
    }
}

bool pieces_of_8(int64_t len, std::initializer_list<const void *> ptrs)
{
    uintptr_t bits = 0;
    for (const void *p : ptrs) bits |= reinterpret_cast<uintptr_t>(p);
    return len % 8 == 0 && (bits & 15) == 0;
}

// F(V) with V = 8 or 1 elements a piece
template <class F>
hipError_t by_piece(bool v8, F &&f)
{
    if (v8) f(std::integral_constant<int, 8>{});
    else f(std::integral_constant<int, 1>{});
    return hipGetLastError();
}

// Workgroups of `per` units each for n units; the kernels stride over what a
// grid of the largest size leaves.
dim3 grid_of(int64_t n, int per = kThreads)
{
    const int64_t g = (n + per - 1) / per;
    return dim3((uint32_t)(g < (1 << 22) ? g : (1 << 22)));
}

const uint16_t *in(const void *p) { return static_cast<const uint16_t *>(p); }
uint16_t *to(void *p) { return static_cast<uint16_t *>(p); }

}  // namespace

hipError_t launch_swiglu(const void *H, void *A, int64_t M, int64_t F, hipStream_t stream)
{
    return by_piece(pieces_of_8(F, {H, A}), [&](auto v) {
        constexpr int V = decltype(v)::value;
        hipLaunchKernelGGL((swiglu_kernel<V>), grid_of(M * F / V), dim3(kThreads), 0, stream, in(H), to(A), M * F / V, F);
    });
}

hipError_t launch_swiglu_bwd(const void *dA, const void *H, void *dH, int64_t M, int64_t F, hipStream_t stream)
{
    return by_piece(pieces_of_8(F, {dA, H, dH}), [&](auto v) {
        constexpr int V = decltype(v)::value;
        hipLaunchKernelGGL((swiglu_bwd_kernel<V>), grid_of(M * F / V), dim3(kThreads), 0, stream, in(dA), in(H), to(dH),
                           M * F / V, F);
    });
}

hipError_t launch_moe_combine(const void *Y, const int32_t *slots, const float *weights, void *out, int64_t T,
                              int64_t M, int k, int64_t H, hipStream_t stream)
{
    return by_piece(pieces_of_8(H, {Y, out}), [&](auto v) {
        constexpr int V = decltype(v)::value;
        hipLaunchKernelGGL((combine_kernel<V>), grid_of(T * H / V), dim3(kThreads), 0, stream, in(Y), slots, weights,
                           to(out), T * H / V, M, k, H);
    });
}

hipError_t launch_moe_combine_bwd(const void *dO, const void *Y, const int32_t *slots, const float *weights,
                                  const int32_t *total, void *dY, float *dweights, int64_t T, int64_t M, int k,
                                  int64_t H, hipStream_t stream)
{
    const dim3 grid = grid_of(T * k, kThreads / 64);
    return by_piece(pieces_of_8(H, {dO, Y, dY}), [&](auto v) {
        constexpr int V = decltype(v)::value;
        hipLaunchKernelGGL((combine_bwd_kernel<V>), grid, dim3(kThreads), 0, stream, in(dO), in(Y), slots, weights,
                           total, to(dY), dweights, T * k, M, k, H);
    });
}

}  // namespace dbs
