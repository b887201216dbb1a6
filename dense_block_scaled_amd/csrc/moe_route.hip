// moe_route.hip -- gfx950 kernels of the mixture-of-experts router.
//
//     w[t, :] = softmax(logits[t, :])       (fp32)
//     experts[t, 0 .. k-1]                  the k largest logits, ties to the lower index
//     weights[t, j]                         w at those experts, or renormalised over them
//
// and the stable order of the T k pairs (t, j) by expert.  A logit of -inf or
// NaN closes an expert to the token; a token with fewer than k open experts
// has experts -1 (weight 0) behind them, and such pairs have no place in the
// order.  +inf counts as the largest finite value.
//
// Selection.  16 lanes hold one token's logits in registers (lane l: experts
// l, 16 + l, ...), so the cross-lane steps of a maximum are four DPP moves
// inside a row of 16 and one wave works on four tokens: at 128 experts eight
// logits a lane, about a hundred vector instructions a token.
//
// Order.  A token's experts are distinct, so inside a workgroup's 64 tokens
// the pairs of one expert, in pair order, are its tokens in token order: an
// expert's 64-bit mask of the tokens that chose it (one LDS or each, in any
// order the same word) holds its count (a population count) and every pair's
// rank (a population count of the bits below the token's).  No rank depends
// on the order of atomics, so results repeat bit for bit.  More than 64
// tokens take three kernels: selection with the counts of each 64 tokens; an
// exclusive sum down every expert's column of counts; and the placing, where
// every workgroup sums the expert totals for itself.  Up to 64 tokens take
// one kernel, which is what a decoding step's latency asks for.
#include <hip/hip_runtime.h>
#include <float.h>
#include <stdint.h>

#include <type_traits>

#include "moe.h"

namespace dbs {
namespace {

constexpr int kThreads = 256;
constexpr int kLanes = 16;                       // lanes per token

// xor-style moves inside a row of 16 lanes; together they reach all of them
template <int STEP, typename V>
__device__ __forceinline__ V row_move(V v)
{
    constexpr int ctrl = STEP == 0 ? 0xB1 : STEP == 1 ? 0x4E : STEP == 2 ? 0x141 : 0x140;
    return __builtin_bit_cast(V, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), ctrl, 0xF, 0xF, true));
}

__device__ __forceinline__ float row_sum(float v)
{
    v += row_move<0>(v);
    v += row_move<1>(v);
    v += row_move<2>(v);
    return v + row_move<3>(v);
}

__device__ __forceinline__ float row_max(float v)
{
    v = fmaxf(v, row_move<0>(v));
    v = fmaxf(v, row_move<1>(v));
    v = fmaxf(v, row_move<2>(v));
    return fmaxf(v, row_move<3>(v));
}

template <int STEP>
__device__ __forceinline__ void best_step(float &v, int &e)
{
    const float ov = row_move<STEP>(v);
    const int oe = row_move<STEP>(e);
    const bool take = ov > v || (ov == v && oe < e);
    v = take ? ov : v;
    e = take ? oe : e;
}

// -inf for a closed expert, at most the largest finite value otherwise
__device__ __forceinline__ float open_logit(float x) { return x == x ? fminf(x, FLT_MAX) : -INFINITY; }

template <bool BF16>
__device__ __forceinline__ float load_logit(const void *logits, int64_t i)
{
    if constexpr (BF16)
        return __builtin_bit_cast(float, (uint32_t) reinterpret_cast<const uint16_t *>(logits)[i] << 16);
    else
        return reinterpret_cast<const float *>(logits)[i];
}

// The exclusive sum of total[0 .. E-1] into base[0 .. E] (LDS), by the whole
// workgroup: thread i sums experts 4 i .. 4 i + 3.
__device__ __forceinline__ void scan_experts(const int32_t *total, int E, int32_t *base, int32_t *part)
{
    static_assert(kMoeMaxExperts <= 4 * kThreads, "four experts a thread");
    const int t = threadIdx.x, lane = t & 63, w = t >> 6;
    int v[4], s = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int e = 4 * t + i;
        v[i] = e < E ? total[e] : 0;
        s += v[i];
    }
    int inc = s;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int o = __shfl_up(inc, d);
        if (lane >= d) inc += o;
    }
    if (lane == 63) part[w] = inc;
    __syncthreads();
    int pre = inc - s;
    for (int i = 0; i < w; ++i) pre += part[i];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int e = 4 * t + i;
        if (e < E) base[e] = pre;
        pre += v[i];
        if (e == E - 1) base[E] = pre;
    }
    __syncthreads();
}

// slots and rows of the workgroup's pairs p0 .. p1-1 (tokens t0 ..), from the
// masks of its tokens, the experts' first rows and the counts of the
// workgroups before it; rows past the last placed pair are -1.
__device__ __forceinline__ void place(const MoeRoute &p, int64_t t0, int64_t p0, int64_t p1, const uint64_t *mask,
                                      const int32_t *base, const int32_t *before, const int32_t *experts)
{
    const int total = base[p.E];
    for (int64_t q = p0 + threadIdx.x; q < p1; q += kThreads) {
        const int64_t t = q / p.k;
        const int e = experts[q - p0];
        int slot = -1;
        if (e >= 0) {
            const uint64_t below = ((uint64_t)1 << (t - t0)) - 1;
            slot = base[e] + (before ? before[e] : 0) + __popcll(mask[e] & below);
            p.rows[slot] = (int32_t)t;
        }
        p.slots[q] = slot;
        if (q >= total) p.rows[q] = -1;
    }
}

// VPL logits per lane (E <= 16 VPL).  ONE: the whole call in this kernel (T <= kRouteTokens).
template <int VPL, bool BF16, bool ONE>
__global__ __launch_bounds__(kThreads) void route_select(MoeRoute p)
{
    __shared__ uint64_t mask[16 * VPL];
    __shared__ int32_t chosen[ONE ? kRouteTokens * kMoeMaxK : 1];
    __shared__ int32_t base[ONE ? 16 * VPL + 1 : 1];
    __shared__ int32_t part[kThreads / 64];
    const int t = threadIdx.x, l = t & (kLanes - 1);
    for (int e = t; e < p.E; e += kThreads) mask[e] = 0;
    __syncthreads();

    const int64_t t0 = (int64_t)blockIdx.x * kRouteTokens;
    for (int tl = t / kLanes; tl < kRouteTokens; tl += kThreads / kLanes) {
        const int64_t tok = t0 + tl;
        if (tok >= p.T) break;                   // (uniform in the token's 16 lanes)
        float v[VPL];
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const int e = 16 * i + l;
            v[i] = e < p.E ? open_logit(load_logit<BF16>(p.logits, tok * p.E + e)) : -INFINITY;
        }
        float mine = -INFINITY, top = 0.0f, whole = 0.0f;   // lane j: the j-th choice
        int mine_e = -1;
        for (int j = 0; j < p.k; ++j) {
            float b = -INFINITY;
            int be = 1 << 30;
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                const bool take = v[i] > b;      // experts of a lane ascend: a tie keeps the lower
                b = take ? v[i] : b;
                be = take ? 16 * i + l : be;
            }
            best_step<0>(b, be);
            best_step<1>(b, be);
            best_step<2>(b, be);
            best_step<3>(b, be);
            if (b == -INFINITY) break;           // no open expert is left
            if (j == 0) {
                top = b;
                if (!p.renorm) {
#pragma unroll
                    for (int i = 0; i < VPL; ++i) whole += expf(v[i] - top);
                    whole = row_sum(whole);
                }
            }
            if (l == j) {
                mine = b;
                mine_e = be;
            }
#pragma unroll
            for (int i = 0; i < VPL; ++i) v[i] = be == 16 * i + l ? -INFINITY : v[i];
        }
        const float x = mine_e >= 0 ? expf(mine - top) : 0.0f;
        if (p.renorm) whole = row_sum(x);
        if (l < p.k) {
            p.experts[tok * p.k + l] = mine_e;
            p.weights[tok * p.k + l] = mine_e >= 0 ? x / whole : 0.0f;
            if (mine_e >= 0) atomicOr(reinterpret_cast<unsigned long long *>(&mask[mine_e]), 1ull << tl);
            if constexpr (ONE) chosen[tl * p.k + l] = mine_e;
        }
    }
    __syncthreads();
    if constexpr (ONE) {
        // the counts (p.counts is not used) in LDS, summed in place of the totals
        for (int e = t; e < p.E; e += kThreads) base[e] = __popcll(mask[e]);
        __syncthreads();
        int32_t *b = base;
        scan_experts(b, p.E, b, part);
        for (int e = t; e <= p.E; e += kThreads) p.offsets[e] = base[e];
        place(p, 0, 0, p.T * p.k, mask, base, nullptr, chosen);
    } else {
        for (int e = t; e < p.E; e += kThreads) p.counts[(int64_t)blockIdx.x * p.E + e] = __popcll(mask[e]);
    }
}

// Exclusive sums down the columns of counts (nb rows of E), in place, and the
// column totals behind them: 16 columns a workgroup, 64 segments of rows.
__global__ __launch_bounds__(1024) void route_columns(int32_t *counts, int64_t nb, int E)
{
    __shared__ int32_t seg[64][17];
    const int col = threadIdx.x & 15, s = threadIdx.x >> 4;
    const int e = blockIdx.x * 16 + col;
    const int64_t per = (nb + 63) / 64, r0 = s * per, r1 = r0 + per < nb ? r0 + per : nb;
    int sum = 0;
    if (e < E)
        for (int64_t r = r0; r < r1; ++r) sum += counts[r * E + e];
    seg[s][col] = sum;
    __syncthreads();
    if (threadIdx.x < 16) {
        int run = 0;
        for (int i = 0; i < 64; ++i) {
            const int v = seg[i][threadIdx.x];
            seg[i][threadIdx.x] = run;
            run += v;
        }
        if (blockIdx.x * 16 + (int)threadIdx.x < E) counts[nb * E + blockIdx.x * 16 + threadIdx.x] = run;
    }
    __syncthreads();
    if (e < E) {
        int run = seg[s][col];
        for (int64_t r = r0; r < r1; ++r) {
            const int v = counts[r * E + e];
            counts[r * E + e] = run;
            run += v;
        }
    }
}

__global__ __launch_bounds__(kThreads) void route_place(MoeRoute p, int64_t nb)
{
    __shared__ uint64_t mask[kMoeMaxExperts];
    __shared__ int32_t base[kMoeMaxExperts + 1];
    __shared__ int32_t chosen[kRouteTokens * kMoeMaxK];
    __shared__ int32_t part[kThreads / 64];
    const int t = threadIdx.x;
    for (int e = t; e < p.E; e += kThreads) mask[e] = 0;
    scan_experts(p.counts + nb * p.E, p.E, base, part);     // (ends with a barrier)
    if (blockIdx.x == 0)
        for (int e = t; e <= p.E; e += kThreads) p.offsets[e] = base[e];
    const int64_t t0 = (int64_t)blockIdx.x * kRouteTokens;
    const int64_t p0 = t0 * p.k, p1 = (t0 + kRouteTokens < p.T ? t0 + kRouteTokens : p.T) * p.k;
    for (int64_t q = p0 + t; q < p1; q += kThreads) {
        const int e = p.experts[q];
        chosen[q - p0] = e;
        if (e >= 0) atomicOr(reinterpret_cast<unsigned long long *>(&mask[e]), 1ull << (q / p.k - t0));
    }
    __syncthreads();
    place(p, t0, p0, p1, mask, base, p.counts + (int64_t)blockIdx.x * p.E, chosen);
}

// dlogits = p (u - sum p u): p the softmax over all experts, or over the
// chosen ones (renorm), u the weights' gradients at the chosen experts and 0
// elsewhere.  16 lanes a token, as in route_select.
template <int VPL, bool BF16>
__global__ __launch_bounds__(kThreads) void route_bwd(const void *logits, int64_t T, int E, int k, int renorm,
                                                      const int32_t *experts, const float *dweights, void *dlogits)
{
    const int l = threadIdx.x & (kLanes - 1);
    const int64_t tok = (int64_t)blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes;
    if (tok >= T) return;                        // (uniform in the token's 16 lanes)
    float v[VPL], u[VPL];
    bool sel[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const int e = 16 * i + l;
        v[i] = e < E ? open_logit(load_logit<BF16>(logits, tok * E + e)) : -INFINITY;
        u[i] = 0.0f;
        sel[i] = false;
    }
    for (int j = 0; j < k; ++j) {
        const int e = experts[tok * k + j];
        const float d = dweights[tok * k + j];
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const bool hit = e == 16 * i + l;
            u[i] = hit ? d : u[i];
            sel[i] = sel[i] || hit;
        }
    }
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        if (renorm && !sel[i]) v[i] = -INFINITY;
        top = fmaxf(top, v[i]);
    }
    top = row_max(top);
    const bool open = top > -INFINITY;           // a closed token has gradient 0
    float sum = 0.0f, dot = 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        v[i] = open ? expf(v[i] - top) : 0.0f;
        sum += v[i];
        dot += v[i] * u[i];
    }
    sum = row_sum(sum);
    dot = row_sum(dot);
    const float inv = open ? 1.0f / sum : 0.0f;
    dot *= inv;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const int e = 16 * i + l;
        if (e >= E) continue;
        const float d = v[i] > 0.0f ? v[i] * inv * (u[i] - dot) : 0.0f;
        if constexpr (BF16)
            reinterpret_cast<__bf16 *>(dlogits)[tok * E + e] = (__bf16)d;
        else
            reinterpret_cast<float *>(dlogits)[tok * E + e] = d;
    }
}

// F(VPL) for the smallest number of logits per lane that holds E experts
template <class F>
hipError_t by_experts(int E, F &&f)
{
    if (E <= 16) return f(std::integral_constant<int, 1>{});
    if (E <= 32) return f(std::integral_constant<int, 2>{});
    if (E <= 64) return f(std::integral_constant<int, 4>{});
    if (E <= 128) return f(std::integral_constant<int, 8>{});
    if (E <= 256) return f(std::integral_constant<int, 16>{});
    if (E <= 512) return f(std::integral_constant<int, 32>{});
    return f(std::integral_constant<int, 64>{});
}

int64_t blocks_of(int64_t T) { return (T + kRouteTokens - 1) / kRouteTokens; }

}  // namespace

int64_t moe_route_workspace_bytes(int64_t T, int64_t E)
{
    return T <= kRouteTokens ? 0 : (blocks_of(T) + 1) * E * (int64_t)sizeof(int32_t);
}

hipError_t launch_moe_route(const MoeRoute &p, hipStream_t stream)
{
    const int64_t nb = blocks_of(p.T);
    const bool one = p.T <= kRouteTokens;
    hipError_t e = by_experts(p.E, [&](auto v) {
        constexpr int V = decltype(v)::value;
        if (one) {
            if (p.bf16) hipLaunchKernelGGL((route_select<V, true, true>), dim3(1), dim3(kThreads), 0, stream, p);
            else hipLaunchKernelGGL((route_select<V, false, true>), dim3(1), dim3(kThreads), 0, stream, p);
        } else {
            if (p.bf16) hipLaunchKernelGGL((route_select<V, true, false>), dim3(nb), dim3(kThreads), 0, stream, p);
            else hipLaunchKernelGGL((route_select<V, false, false>), dim3(nb), dim3(kThreads), 0, stream, p);
        }
        return hipGetLastError();
    });
    if (e != hipSuccess || one) return e;
    hipLaunchKernelGGL(route_columns, dim3((p.E + 15) / 16), dim3(1024), 0, stream, p.counts, nb, p.E);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    hipLaunchKernelGGL(route_place, dim3(nb), dim3(kThreads), 0, stream, p, nb);
    return hipGetLastError();
}

hipError_t launch_moe_route_bwd(const void *logits, int bf16, int64_t T, int E, int k, int renorm,
                                const int32_t *experts, const float *dweights, void *dlogits, hipStream_t stream)
{
    const dim3 grid((T + kThreads / kLanes - 1) / (kThreads / kLanes));
    return by_experts(E, [&](auto v) {
        constexpr int V = decltype(v)::value;
        if (bf16)
            hipLaunchKernelGGL((route_bwd<V, true>), grid, dim3(kThreads), 0, stream, logits, T, E, k, renorm, experts,
                               dweights, dlogits);
        else
            hipLaunchKernelGGL((route_bwd<V, false>), grid, dim3(kThreads), 0, stream, logits, T, E, k, renorm, experts,
                               dweights, dlogits);
        return hipGetLastError();
    });
}

}  // namespace dbs
