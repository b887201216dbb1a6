// moe_route.hip -- gfx950 kernels of the mixture-of-experts router.
//
//     w[t, :] = softmax(logits[t, :])       (fp32)
//     experts[t, 0 .. k-1]                  the k largest logits, ties to the lower index
//     weights[t, j]                         w at those experts, or renormalised over them
//
// and the stable order of the T k pairs (t, j) by expert.  A logit of -inf or
// NaN closes an expert to the token; a token with fewer than k open experts
// has experts -1 (weight 0) behind them, and such pairs have no place in the
// order.  +inf counts as the largest finite fp32 value.
//
// Selection.  16 lanes hold one token's logits in registers, so the
// cross-lane steps of a maximum are four DPP moves inside a row of 16 and one
// wave works on four tokens: for every choice the largest value, the lowest
// expert that has it, and that one struck out.
//
// Order.  A token's experts are distinct, so inside a workgroup's 64 tokens
// the pairs of one expert, in pair order, are its tokens in token order: an
// expert's 64-bit mask of the tokens that chose it (one LDS or each, in any
// order the same word) holds its count (a population count) and every pair's
// rank (a population count of the bits below the token's).  No rank depends
// on the order of atomics, so results repeat bit for bit.  More than 64
// tokens take three kernels: selection with the counts of each 64 tokens; an
// exclusive sum down every expert's column of counts; and the placing, where
// every workgroup sums the expert totals for itself -- and, up to 2048 tokens,
// the columns too, so that two kernels do.  Up to 64 tokens take one kernel,
// which is what a decoding step's latency asks for: one token of 64 experts
// 3.6 us, nearly all of it the launch and two trips to memory.
//
// 32768 tokens, 8 of 128 experts, fp32: 11.5 us of selection, 4.1 of sums and 5.5
// of placing, for 21 MB.  Selection is bound by its vector instructions (73 a
// choice and wave of four tokens, 9 us of issue on 1024 SIMDs), not by the
// logits (1.4 TB/s).  The gradient streams: 16384 tokens of 160 experts, bf16,
// 6.1 us (1.9 TB/s).
#include <hip/hip_runtime.h>
#include <float.h>
#include <stdint.h>

#include <type_traits>

#include "moe.h"
#include "moe_device.h"

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

__device__ __forceinline__ int row_min(int v)
{
    v = min(v, row_move<0>(v));
    v = min(v, row_move<1>(v));
    v = min(v, row_move<2>(v));
    return min(v, row_move<3>(v));
}

// -inf for a closed expert, at most the largest finite value otherwise
__device__ __forceinline__ float open_logit(float x) { return x == x ? fminf(x, FLT_MAX) : -INFINITY; }

// How a token's experts lie in its 16 lanes: C consecutive ones a lane and
// step, so value i of lane l is expert 16 C (i / C) + C l + i % C.  C = 4
// (whole loads of 8 or 16 bytes) where the rows of logits allow it, else 1.
template <int C>
__device__ __forceinline__ int expert_of(int i, int l) { return (i / C) * 16 * C + C * l + i % C; }

template <int VPL, int C, bool BF16>
__device__ __forceinline__ void load_logits(float (&v)[VPL], const void *logits, int64_t tok, int E, int l)
{
    typedef __attribute__((ext_vector_type(4))) float f32x4;
    typedef __attribute__((ext_vector_type(2))) uint32_t u32x2;
#pragma unroll
    for (int i = 0; i < VPL; i += C) {
        const int e = expert_of<C>(i, l);
        float x[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        if (e < E) {                             // (E is a multiple of C)
            const int64_t at = tok * E + e;
            if constexpr (BF16 && C == 4) {
                const u32x2 w = *reinterpret_cast<const u32x2 *>(reinterpret_cast<const uint16_t *>(logits) + at);
                x[0] = __builtin_bit_cast(float, w[0] << 16);
                x[1] = __builtin_bit_cast(float, w[0] & 0xFFFF0000u);
                x[2] = __builtin_bit_cast(float, w[1] << 16);
                x[3] = __builtin_bit_cast(float, w[1] & 0xFFFF0000u);
            } else if constexpr (BF16) {
                x[0] = __builtin_bit_cast(float, (uint32_t) reinterpret_cast<const uint16_t *>(logits)[at] << 16);
            } else if constexpr (C == 4) {
                const f32x4 w = *reinterpret_cast<const f32x4 *>(reinterpret_cast<const float *>(logits) + at);
#pragma unroll
                for (int c = 0; c < 4; ++c) x[c] = w[c];
            } else {
                x[0] = reinterpret_cast<const float *>(logits)[at];
            }
        }
#pragma unroll
        for (int c = 0; c < C; ++c) v[i + c] = open_logit(x[c]);
    }
}

// The exclusive sum of total[0 .. E-1] into base[0 .. E] (LDS), by the whole
// workgroup: thread i sums experts 4 i .. 4 i + 3.
__device__ __forceinline__ void scan_experts(const int32_t *total, int E, int32_t *base, int32_t *part)
{
    static_assert(kMoeMaxExperts <= 4 * 256, "four experts a thread");
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
    for (int64_t q = p0 + threadIdx.x; q < p1; q += blockDim.x) {
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

// VPL logits per lane (E <= 16 VPL).  ONE: the whole call in this kernel (T <=
// kRouteTokens); otherwise every token of the workgroup has lanes of its own
// (up to 512 experts), which puts eight waves on a SIMD from 32768 tokens on.
template <int VPL, bool ONE>
constexpr int select_threads() { return ONE ? 256 : VPL > 32 ? 512 : 1024; }

template <int VPL, int C, bool BF16, bool ONE>
__global__ __launch_bounds__((select_threads<VPL, ONE>())) void route_select(MoeRoute p)
{
    __shared__ uint64_t mask[16 * VPL];
    __shared__ int32_t chosen[ONE ? kRouteTokens * kMoeMaxK : 1];
    __shared__ int32_t base[ONE ? 16 * VPL + 1 : 1];
    __shared__ int32_t part[4];
    constexpr int kThreads = select_threads<VPL, ONE>();
    const int t = threadIdx.x, l = t & (kLanes - 1);
    for (int e = t; e < p.E; e += kThreads) mask[e] = 0;
    __syncthreads();

    const int64_t t0 = (int64_t)blockIdx.x * kRouteTokens;
    for (int tl = t / kLanes; tl < kRouteTokens; tl += kThreads / kLanes) {
        const int64_t tok = t0 + tl;
        if (tok >= p.T) break;                   // (uniform in the token's 16 lanes)
        float v[VPL];
        load_logits<VPL, C, BF16>(v, p.logits, tok, p.E, l);
        float mine = -INFINITY, top = 0.0f, whole = 0.0f;   // lane j: the j-th choice
        int mine_e = -1;
        for (int j = 0; j < p.k; ++j) {
            // the largest value, then the lowest expert that has it
            float b = v[0];
#pragma unroll
            for (int i = 1; i < VPL; ++i) b = fmaxf(b, v[i]);
            b = row_max(b);
            if (b == -INFINITY) break;           // no open expert is left
            int be = 1 << 30;
#pragma unroll
            for (int i = VPL - 1; i >= 0; --i) be = v[i] == b ? expert_of<C>(i, l) : be;
            be = row_min(be);
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
            for (int i = 0; i < VPL; ++i) v[i] = be == expert_of<C>(i, l) ? -INFINITY : v[i];
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
        // the counts in LDS, summed in place
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
    if (e < E) {
#pragma unroll 8
        for (int64_t r = r0; r < r1; ++r) sum += counts[r * E + e];
    }
    seg[s][col] = sum;
    __syncthreads();
    {
        // a wave per column, a lane per segment
        const int lane = threadIdx.x & 63, c = threadIdx.x >> 6, v = seg[lane][c];
        int inc = v;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const int o = __shfl_up(inc, d);
            if (lane >= d) inc += o;
        }
        seg[lane][c] = inc - v;
        if (lane == 63 && blockIdx.x * 16 + c < E) counts[nb * E + blockIdx.x * 16 + c] = inc;
    }
    __syncthreads();
    if (e < E) {
        int run = seg[s][col];
#pragma unroll 8
        for (int64_t r = r0; r < r1; ++r) {
            const int v = counts[r * E + e];
            counts[r * E + e] = run;
            run += v;
        }
    }
}

// DIRECT: every workgroup sums the columns for itself (up to kDirect rows of
// counts), which leaves out the kernel before.
template <bool DIRECT>
__global__ __launch_bounds__(kThreads) void route_place(MoeRoute p, int64_t nb)
{
    __shared__ uint64_t mask[kMoeMaxExperts];
    __shared__ int32_t base[kMoeMaxExperts + 1];
    __shared__ int32_t before[DIRECT ? kMoeMaxExperts : 1], total[DIRECT ? kMoeMaxExperts : 1];
    __shared__ int32_t chosen[kRouteTokens * kMoeMaxK];
    __shared__ int32_t part[kThreads / 64];
    const int t = threadIdx.x;
    for (int e = t; e < p.E; e += kThreads) {
        mask[e] = 0;
        if constexpr (DIRECT) {
            int mine = 0, all = 0;
#pragma unroll 8
            for (int r = 0; r < (int)nb; ++r) {
                const int v = p.counts[(int64_t)r * p.E + e];
                mine += r < (int)blockIdx.x ? v : 0;
                all += v;
            }
            before[e] = mine;
            total[e] = all;
        }
    }
    if constexpr (DIRECT) __syncthreads();
    const int32_t *totals = DIRECT ? total : p.counts + nb * p.E;
    scan_experts(totals, p.E, base, part);                  // (ends with a barrier)
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
    place(p, t0, p0, p1, mask, base, DIRECT ? before : p.counts + (int64_t)blockIdx.x * p.E, chosen);
}

// dlogits = p (u - sum p u): p the softmax over all experts, or over the
// chosen ones (renorm), u the weights' gradients at the chosen experts and 0
// elsewhere.  16 lanes a token, as in route_select; lane j has the j-th
// choice, and the chosen experts' gradients reach the lanes that hold those
// experts through a row of E floats in LDS (zeroed, written and read by the
// token's own lanes of one wave, with a handover between).
template <int VPL, int C, bool BF16>
__global__ __launch_bounds__(kThreads) void route_bwd(const void *logits, int64_t T, int E, int k, int renorm,
                                                      const int32_t *experts, const float *dweights, void *dlogits)
{
    // lane l's values lie together, C at a time: [token][i / C][l][i % C]
    __shared__ __attribute__((aligned(16))) float at_chosen[kThreads / kLanes][16 * VPL];
    const int l = threadIdx.x & (kLanes - 1);
    const int64_t tok = (int64_t)blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes;
    if (tok >= T) return;                        // (uniform in the token's 16 lanes)
    float *row = at_chosen[threadIdx.x / kLanes];
    float v[VPL];
    load_logits<VPL, C, BF16>(v, logits, tok, E, l);
    int e = -1;
    float u = 0.0f, x = -INFINITY;
    if (l < k) {
        e = experts[tok * k + l];
        e = e < E ? e : -1;
        if (e >= 0) {
            u = dweights[tok * k + l];
            const int64_t at = tok * E + e;
            if constexpr (BF16)
                x = open_logit(__builtin_bit_cast(float, (uint32_t) reinterpret_cast<const uint16_t *>(logits)[at] << 16));
            else
                x = open_logit(reinterpret_cast<const float *>(logits)[at]);
        }
    }
    // the softmax's maximum and sum, over all experts or the chosen ones
    float top = x;
    if (!renorm) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) top = fmaxf(top, v[i]);
    }
    top = row_max(top);
    const bool open = top > -INFINITY;           // a closed token has gradient 0
    float sum = 0.0f;
    const float mine = open ? expf(x - top) : 0.0f;
    if (renorm) {
        sum = mine;
    } else {
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            v[i] = open ? expf(v[i] - top) : 0.0f;
            sum += v[i];
        }
    }
    const float inv = open ? 1.0f / row_sum(sum) : 0.0f;
    const float p = mine * inv, dot = row_sum(p * u);
    const float scale = renorm ? 0.0f : dot * inv;
#pragma unroll
    for (int i = 0; i < VPL; ++i) row[expert_of<C>(i, l)] = 0.0f;
    wave_handover();
    if (e >= 0) row[e] = renorm ? p * (u - dot) : p * u;
    wave_handover();
#pragma unroll
    for (int i = 0; i < VPL; i += C) {
        const int first = expert_of<C>(i, l);
        if (first >= E) continue;
        float d[C];
#pragma unroll
        for (int c = 0; c < C; ++c) d[c] = renorm ? row[first + c] : row[first + c] - v[i + c] * scale;
        const int64_t at = tok * E + first;
        if constexpr (BF16) {
            __bf16 w[C];
#pragma unroll
            for (int c = 0; c < C; ++c) w[c] = (__bf16)d[c];
            __builtin_memcpy(reinterpret_cast<__bf16 *>(dlogits) + at, w, sizeof(w));
        } else {
            __builtin_memcpy(reinterpret_cast<float *>(dlogits) + at, d, sizeof(d));
        }
    }
}

// F(VPL, C) for the smallest number of logits per lane that holds E experts;
// C = 4 if every row starts on a whole load and ends with one.
template <class F>
hipError_t by_experts(int E, const void *logits, const void *other, F &&f)
{
    const bool whole = E % 4 == 0 && ((reinterpret_cast<uintptr_t>(logits) | reinterpret_cast<uintptr_t>(other)) & 15) == 0;
    auto with = [&](auto v) {
        return whole ? f(v, std::integral_constant<int, 4>{}) : f(v, std::integral_constant<int, 1>{});
    };
    if (E <= 64) return with(std::integral_constant<int, 4>{});
    if (E <= 128) return with(std::integral_constant<int, 8>{});
    if (E <= 192) return with(std::integral_constant<int, 12>{});
    if (E <= 256) return with(std::integral_constant<int, 16>{});
    if (E <= 512) return with(std::integral_constant<int, 32>{});
    return with(std::integral_constant<int, 64>{});
}

// Rows of counts up to which the placing workgroups sum them for themselves.
constexpr int kDirect = 32;

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
    hipError_t e = by_experts(p.E, p.logits, nullptr, [&](auto vpl, auto c) {
        constexpr int V = decltype(vpl)::value, C = decltype(c)::value;
        if (one) {
            if (p.bf16) hipLaunchKernelGGL((route_select<V, C, true, true>), dim3(1), dim3(256), 0, stream, p);
            else hipLaunchKernelGGL((route_select<V, C, false, true>), dim3(1), dim3(256), 0, stream, p);
        } else {
            if (p.bf16) hipLaunchKernelGGL((route_select<V, C, true, false>), dim3(nb), dim3(select_threads<V, false>()), 0, stream, p);
            else hipLaunchKernelGGL((route_select<V, C, false, false>), dim3(nb), dim3(select_threads<V, false>()), 0, stream, p);
        }
        return hipGetLastError();
    });
    if (e != hipSuccess || one) return e;
    if (nb <= kDirect) {
        hipLaunchKernelGGL((route_place<true>), dim3(nb), dim3(kThreads), 0, stream, p, nb);
        return hipGetLastError();
    }
    hipLaunchKernelGGL(route_columns, dim3((p.E + 15) / 16), dim3(1024), 0, stream, p.counts, nb, p.E);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    hipLaunchKernelGGL((route_place<false>), dim3(nb), dim3(kThreads), 0, stream, p, nb);
    return hipGetLastError();
}

hipError_t launch_moe_route_bwd(const void *logits, int bf16, int64_t T, int E, int k, int renorm,
                                const int32_t *experts, const float *dweights, void *dlogits, hipStream_t stream)
{
    const dim3 grid((T + kThreads / kLanes - 1) / (kThreads / kLanes));
    return by_experts(E, logits, dlogits, [&](auto vpl, auto c) {
        constexpr int V = decltype(vpl)::value, C = decltype(c)::value;
        if (bf16)
            hipLaunchKernelGGL((route_bwd<V, C, true>), grid, dim3(kThreads), 0, stream, logits, T, E, k, renorm,
                               experts, dweights, dlogits);
        else
            hipLaunchKernelGGL((route_bwd<V, C, false>), grid, dim3(kThreads), 0, stream, logits, T, E, k, renorm,
                               experts, dweights, dlogits);
        return hipGetLastError();
    });
}

}  // namespace dbs
