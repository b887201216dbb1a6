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
    // (a workgroup's pairs are few: 32 bits, whose division is short)
    for (uint32_t i = threadIdx.x; i < (uint32_t)(p1 - p0); i += blockDim.x) {
        const uint32_t tl = i / (uint32_t)p.k;
        const int64_t q = p0 + i, t = t0 + tl;
        const int e = experts[i];
        int slot = -1;
        if (e >= 0) {
            const uint64_t below = ((uint64_t)1 << tl) - 1;
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

// ------------------------------------------------------- selection by groups
//
//     s_e = sigmoid(logits[t, e])  or  softmax(logits[t, :])_e
//     c_e = s_e + bias_e                     what the choice goes by
//     group's score                          the sum of its best one or two c
//     experts[t, 0 .. k-1]                   the k largest c of the kept groups with the largest scores
//     weights[t, j]                          scale s at those experts, or scale s / (the sum of s over them)
//
// Choices must not hang on a rounding: c is computed in fp64 (vector fp64 runs at
// fp32's rate here).  The expert's index lies in the ten lowest bits of
// its c, so keys differ, ties go to the lower index, and sorting needs no second
// register: two instructions for every exchange of a lane's network.  After the sort a lane's best are its
// first, groups' sums come from neighbouring lanes, and four merges of sorted
// lists leave every lane the token's k best (one maximum over the lanes' heads for
// every choice took 4 us more of 16384 tokens of 256 experts).
//
// How near two c may lie and still be told apart, t the larger of s and |bias| of both: a sigmoid
// is off by 2^-44.8 s (exp64), a softmax score by 2^-42 s (exp64 and the rounding of a difference of
// logits up to 708, 2^-44, both a second time in the sum), and a key drops 2^-42 of c, which is
// at most 2 t.  For two of them 2 2^-42 t + 2^-41 t = 2^-40 t, also where a bias near -s leaves little of c.
// A group's score sums two c and is cut once more, at most 4 t: 4 (2^-42 + 2^-41) t + 2^-40 t = 2^-38 t.
// (The callers are told twice as much.)
//
// One token of 256 experts: 6.6 us, the launch, two trips to memory and one wave's chain
// of instructions.  16384 tokens, 8 of 256 experts in 4 of 8 groups, fp32: 16 us of choice, bound by its
// vector instructions (1500 a wave of four tokens, a third of them the sigmoids';
// 10 us of issue on 1024 SIMDs), and 7.2 of order (route_place_bytes).
//
// Lanes.  The 16 lanes of a token are cut into as many runs as the groups'
// count rounded up to a power of two, one run a group; a lane has Q experts in a
// row (see launch_moe_route_grouped).

template <int STEP>
__device__ __forceinline__ double row_move64(double v)
{
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = row_move<STEP>((uint32_t)b), hi = row_move<STEP>((uint32_t)(b >> 32));
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

__device__ __forceinline__ double row_sum64(double v)
{
    v += row_move64<0>(v);
    v += row_move64<1>(v);
    v += row_move64<2>(v);
    return v + row_move64<3>(v);
}

// e^x for -708 <= x <= 708, off by less than 2^-44.9 of it: x = (n + f) ln 2 with |f| <= 1 / 2, and 2^f as
// the polynomial of degree 9 that agrees with it at the Chebyshev nodes (off by 2^-45.6
// at most; the series needs two terms more for that).  log2(e)'s own rounding adds |x| 2^-55.9 (2^-46.5 at the
// ends); the product with it is rounded nowhere, being part of an fma both times.  n is
// taken from the low bits of a sum with 3 2^51, and put in by adding to the exponent
// (the conversions, v_rndne_f64 and v_ldexp_f64 among them, issue more slowly).
__device__ __forceinline__ double exp64(double x)
{
    constexpr double kRound = 6755399441055744.0;
    constexpr double kLog2e = 1.4426950408889634;
    const double shifted = __builtin_fma(x, kLog2e, kRound);
    const double f = __builtin_fma(x, kLog2e, -(shifted - kRound));
    double p = 1.0205905413765595e-07;
    constexpr double c[9] = {1.325964524488711e-06, 1.5252672924850737e-05, 0.0001540343375125101,
                             0.0013333558200794592, 0.009618129193934313,   0.05550410866465167,
                             0.2402265069564034,    0.6931471805599462,     1.0000000000000135};
#pragma unroll
    for (int i = 0; i < 9; ++i) p = __builtin_fma(p, f, c[i]);
    const uint64_t b = __builtin_bit_cast(uint64_t, p);
    const uint32_t hi = (uint32_t)(b >> 32) + ((uint32_t)__builtin_bit_cast(uint64_t, shifted) << 20);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | (uint32_t)b);
}

// 1 / x, x a normal number: y = v_rcp_f64 is off by a factor of 1 - d, d < 2^-20, and y (1 + d + d^2) by d^3
__device__ __forceinline__ double inverse64(double x)
{
    const double y = __builtin_amdgcn_rcp(x), d = __builtin_fma(-x, y, 1.0);
    return __builtin_fma(y, __builtin_fma(d, d, d), y);
}

constexpr uint64_t kIndexBits = 1023;           // kMoeMaxExperts - 1

// c with index e in its lowest bits: larger for a larger c, then for a lower e
__device__ __forceinline__ double keyed(double c, int e)
{
    const uint64_t b = __builtin_bit_cast(uint64_t, c);
    const uint32_t hi = (uint32_t)(b >> 32), flip = ~(uint32_t)((int32_t)hi >> 31) & (uint32_t)kIndexBits;
    const uint32_t lo = ((uint32_t)b & ~(uint32_t)kIndexBits) | ((uint32_t)e ^ flip);      // e, or 1023 - e
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

__device__ __forceinline__ double unkeyed(double key)
{
    return __builtin_bit_cast(double, __builtin_bit_cast(uint64_t, key) & ~kIndexBits);
}

__device__ __forceinline__ int key_index(double key)
{
    const uint64_t b = __builtin_bit_cast(uint64_t, key);
    const int low = (int)(b & kIndexBits);
    return (int64_t)b < 0 ? low : (int)kIndexBits - low;
}

// Odd-even merge sort of v[0 .. N-1], descending
template <int LO, int N, int R, int VPL>
__device__ __forceinline__ void merge_sorted(double (&v)[VPL])
{
    auto order = [&](int a, int b) {
        const double hi = fmax(v[a], v[b]), lo = fmin(v[a], v[b]);
        v[a] = hi;
        v[b] = lo;
    };
    if constexpr (2 * R < N) {
        merge_sorted<LO, N, 2 * R>(v);
        merge_sorted<LO + R, N, 2 * R>(v);
#pragma unroll
        for (int i = LO + R; i + R < LO + N; i += 2 * R) order(i, i + R);
    } else {
        order(LO, LO + R);
    }
}

template <int LO, int N, int VPL>
__device__ __forceinline__ void sort_down(double (&v)[VPL])
{
    if constexpr (N > 1) {
        sort_down<LO, N / 2>(v);
        sort_down<LO + N / 2, N / 2>(v);
        merge_sorted<LO, N, 1>(v);
    }
}

// A descending list of N in every lane becomes that of the N largest of all 16
// lanes, the same in each: lane by lane the larger of one's list and the
// other's from its end are the N largest of both, falling and rising, which log2 N
// steps of exchanges sort.
template <int STEP, int N, int VPL>
__device__ __forceinline__ void best_of_both(double (&v)[VPL])
{
    double o[N];
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = row_move64<STEP>(v[N - 1 - i]);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = fmax(v[i], o[i]);
#pragma unroll
    for (int d = N / 2; d > 0; d /= 2)
#pragma unroll
        for (int i = 0; i < N; ++i)
            if ((i & d) == 0) {
                const double hi = fmax(v[i], v[i + d]), lo = fmin(v[i], v[i + d]);
                v[i] = hi;
                v[i + d] = lo;
            }
}

template <int N, int VPL>
__device__ __forceinline__ void best_of_row(double (&v)[VPL])
{
    best_of_both<0, N>(v);
    best_of_both<1, N>(v);
    best_of_both<2, N>(v);
    best_of_both<3, N>(v);
}

// How many of the lanes BY, 2 BY .. further on in the row of 16 have a larger value
template <int BY, int AT = BY>
__device__ __forceinline__ int larger_in_row(double v)
{
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_mov_dpp((int)b, 0x120 + AT, 0xF, 0xF, true);               // row_ror
    const uint32_t hi = __builtin_amdgcn_mov_dpp((int)(b >> 32), 0x120 + AT, 0xF, 0xF, true);
    const int n = __builtin_bit_cast(double, (uint64_t)hi << 32 | lo) > v;
    if constexpr (AT + BY < 16) return n + larger_in_row<BY, AT + BY>(v);
    return n;
}

// C consecutive values of an array as fp32: to[i ..]
template <int C, int N>
__device__ __forceinline__ void load_some(float (&to)[N], int i, const float *from)
{
    typedef __attribute__((ext_vector_type(4))) float f32x4;
    if constexpr (C == 4) {
        const f32x4 w = *reinterpret_cast<const f32x4 *>(from);
#pragma unroll
        for (int c = 0; c < 4; ++c) to[i + c] = w[c];
    } else {
        to[i] = *from;
    }
}

template <int C, int N>
__device__ __forceinline__ void load_some(float (&to)[N], int i, const uint16_t *from)
{
    typedef __attribute__((ext_vector_type(2))) uint32_t u32x2;
    if constexpr (C == 4) {
        const u32x2 w = *reinterpret_cast<const u32x2 *>(from);
#pragma unroll
        for (int c = 0; c < 4; ++c)
            to[i + c] = __builtin_bit_cast(float, c & 1 ? w[c >> 1] & 0xFFFF0000u : w[c >> 1] << 16);
    } else {
        to[i] = __builtin_bit_cast(float, (uint32_t)*from << 16);
    }
}

// The experts of a token, chosen by its 16 lanes (l: lane of the 16): lane j
// returns the j-th choice (-1: none) and its weight.  VPL: keys a lane has
// registers for (p.q used); C: as in load_logits.
template <int VPL, int C, bool BF16>
__device__ __forceinline__ void choose(const MoeRouteGrouped &p, int64_t tok, int l, int &expert, float &weight)
{
    const int per = p.r.E / p.groups, group = l / p.lanes, at0 = l % p.lanes * p.q;    // first of the lane's in its group
    const int have = group < p.groups ? max(min(per - at0, p.q), 0) : 0, e0 = have ? group * per + at0 : 0;
    const float *logits32 = reinterpret_cast<const float *>(p.r.logits) + tok * p.r.E;
    const uint16_t *logits16 = reinterpret_cast<const uint16_t *>(p.r.logits) + tok * p.r.E;
    // All loads are under way together: what a lane has no expert for reads its last one's again
    float x[VPL], bias[VPL];
    const int last = max(have - C, 0);           // (C = 4: have is a multiple of 4)
#pragma unroll
    for (int i = 0; i < VPL; i += C) {
        const int e = e0 + min(i, last);
        if constexpr (BF16) load_some<C>(x, i, logits16 + e);
        else load_some<C>(x, i, logits32 + e);
    }
    auto load_bias = [&] {
        if (!p.bias) return;
#pragma unroll
        for (int i = 0; i < VPL; i += C) load_some<C>(bias, i, p.bias + e0 + min(i, last));
    };
    if constexpr (VPL <= 16) load_bias();
#pragma unroll
    for (int i = 0; i < VPL; ++i) x[i] = i < have ? open_logit(x[i]) : -INFINITY;
    float top = 0.0f;
    double whole = 1.0, v[VPL];
    if (p.sigmoid) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) v[i] = inverse64(1.0 + exp64((double)fminf(fmaxf(-x[i], -708.0f), 708.0f)));
    } else {
        top = x[0];
#pragma unroll
        for (int i = 1; i < VPL; ++i) top = fmaxf(top, x[i]);
        top = row_max(top);
        const float from = top > -INFINITY ? top : 0.0f;
        whole = 0.0;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            // (the difference in fp64: it need not be an fp32 number)
            const double d = fmax((double)x[i] - (double)from, -708.0);
            const double e = exp64(d);
            v[i] = x[i] > -INFINITY ? e : 0.0;
            whole += v[i];
        }
        whole = row_sum64(whole);
        const double inv = top > -INFINITY ? inverse64(whole) : 0.0;
#pragma unroll
        for (int i = 0; i < VPL; ++i) v[i] *= inv;
    }
    if constexpr (VPL > 16) load_bias();         // (more of them have no registers until now)
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const float b = p.bias ? open_logit(bias[i]) : 0.0f;
        const double key = keyed(v[i] + (double)b, e0 + i);
        v[i] = fminf(x[i], b) > -INFINITY ? key : -(double)INFINITY;
    }
    sort_down<0, VPL>(v);

    if (p.kept < p.groups) {
        // the group's best two, from its lanes' best two
        double one = v[0], two = v[1];
        auto join = [&](double o1, double o2) {
            two = fmax(fmin(one, o1), fmax(two, o2));
            one = fmax(one, o1);
        };
        if (p.lanes > 1) join(row_move64<0>(one), row_move64<0>(two));
        if (p.lanes > 2) join(row_move64<1>(one), row_move64<1>(two));
        if (p.lanes > 4) join(row_move64<2>(one), row_move64<2>(two));
        double score = -(double)INFINITY;
        if (one > -(double)INFINITY) {
            score = unkeyed(one);
            if (p.best == 2 && two > -(double)INFINITY) score += unkeyed(two);
            score = keyed(score, group);
        }
        // (a group's lanes all have its score; at most 16 groups, at least two: 1 .. 8 lanes)
        const int rank = p.lanes == 1 ? larger_in_row<1>(score) : p.lanes == 2 ? larger_in_row<2>(score)
                       : p.lanes == 4 ? larger_in_row<4>(score) : larger_in_row<8>(score);
        const bool keep = rank < p.kept && one > -(double)INFINITY;
#pragma unroll
        for (int i = 0; i < (VPL < kMoeMaxK ? VPL : kMoeMaxK); ++i) v[i] = keep ? v[i] : -(double)INFINITY;
    }

    // the k best of all lanes, and the lane's own of them
    constexpr int N8 = 8, N16 = 16;
    double w[N16];
#pragma unroll
    for (int i = 0; i < N16; ++i) w[i] = i < VPL ? v[i < VPL ? i : 0] : -(double)INFINITY;
    if (p.r.k <= N8) best_of_row<N8>(w);
    else best_of_row<N16>(w);
    double key = w[0];
#pragma unroll
    for (int i = 1; i < N16; ++i) {
        const double other = w[i];
        key = l == i ? other : key;
    }
    expert = l < p.r.k && key > -(double)INFINITY ? key_index(key) : -1;

    // the weights, from the chosen logits: sigmoid(y) = e^min(y, 0) / (1 + e^-|y|), of which
    // renormalising cancels the largest e^min(y, 0)
    float y = -INFINITY;
    if (expert >= 0) {
        if constexpr (BF16) y = __builtin_bit_cast(float, (uint32_t)logits16[expert] << 16);
        else y = logits32[expert];
        y = open_logit(y);
    }
    float s = 0.0f, from = p.sigmoid ? 0.0f : top;
    if (p.r.renorm) from = row_max(p.sigmoid ? fminf(y, 0.0f) : y);
    if (expert >= 0) s = p.sigmoid ? expf(fminf(y, 0.0f) - from) / (1.0f + expf(-fabsf(y))) : expf(y - from);
    const float total = p.r.renorm ? row_sum(s) : p.sigmoid ? 1.0f : (float)whole;
    weight = expert >= 0 ? s / total * p.scale : 0.0f;
}

// Rows of counts up to which route_choose leaves them as bytes, and such a row's length
constexpr int kBytes = 256;
__host__ __device__ constexpr int byte_row(int E) { return (E + 15) & ~15; }

// As route_select, with the choice above, g.tokens to a workgroup: 16 while the CUs
// are not all taken so (1024 tokens of 256 experts on 16 CUs: 15 us), else more.
template <int VPL, int C, bool BF16, bool ONE, int THREADS>
__global__ __launch_bounds__(THREADS) void route_choose(MoeRouteGrouped g)
{
    __shared__ uint64_t mask[kMoeMaxExperts];
    __shared__ int32_t chosen[ONE ? kRouteTokens * kMoeMaxK : 1];
    __shared__ int32_t base[ONE ? kMoeMaxExperts + 1 : 1];
    __shared__ int32_t part[16];
    const MoeRoute &p = g.r;
    const int t = threadIdx.x, l = t & (kLanes - 1);
    for (int e = t; e < p.E; e += THREADS) mask[e] = 0;
    __syncthreads();
    const int64_t t0 = (int64_t)blockIdx.x * g.tokens;
    // (256 threads are for 16 tokens, so that those and 1024 have one round, which is no loop)
    constexpr int kMost = THREADS == 256 ? 16 : kRouteTokens;
    for (int tl = t / kLanes; tl < kMost; tl += THREADS / kLanes) {
        const int64_t tok = t0 + tl;
        if (tl >= g.tokens || tok >= p.T) break; // (uniform in the token's 16 lanes)
        int e;
        float w;
        choose<VPL, C, BF16>(g, tok, l, e, w);
        if (l < p.k) {
            p.experts[tok * p.k + l] = e;
            p.weights[tok * p.k + l] = w;
            if (e >= 0) atomicOr(reinterpret_cast<unsigned long long *>(&mask[e]), 1ull << tl);
            if constexpr (ONE) chosen[tl * p.k + l] = e;
        }
    }
    __syncthreads();
    if constexpr (ONE) {
        for (int e = t; e < p.E; e += THREADS) base[e] = __popcll(mask[e]);
        __syncthreads();
        int32_t *b = base;
        scan_experts(b, p.E, b, part);
        for (int e = t; e <= p.E; e += THREADS) p.offsets[e] = base[e];
        place(p, 0, 0, p.T * p.k, mask, base, nullptr, chosen);
    } else if (g.bytes) {
        const int row = byte_row(p.E);
        uint8_t *counts = reinterpret_cast<uint8_t *>(p.counts) + (int64_t)blockIdx.x * row;
        for (int e = t; e < row; e += THREADS) counts[e] = e < p.E ? (uint8_t)__popcll(mask[e]) : (uint8_t)0;
    } else {
        for (int e = t; e < p.E; e += THREADS) p.counts[(int64_t)blockIdx.x * p.E + e] = __popcll(mask[e]);
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
        if (e >= 0) atomicOr(reinterpret_cast<unsigned long long *>(&mask[e]), 1ull << ((uint32_t)(q - p0) / (uint32_t)p.k));
    }
    __syncthreads();
    place(p, t0, p0, p1, mask, base, DIRECT ? before : p.counts + (int64_t)blockIdx.x * p.E, chosen);
}

// Up to kBytes rows of counts behind route_choose: they are bytes there (64 tokens
// make at most 64), rows of whole 16-byte pieces, and every workgroup sums all
// of them for itself, two launches in place of three (16384 tokens of 256
// experts: 64 KiB a workgroup, 7.3 us where the two kernels take 9.1 and a launch).  A
// thread sums 16 experts of every so manyth row as pairs of 16-bit numbers, its
// wave's lanes and then the waves meet.
__global__ __launch_bounds__(1024) void route_place_bytes(MoeRoute p, int nb, int tokens)
{
    typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;
    __shared__ uint64_t mask[kMoeMaxExperts];
    __shared__ int32_t base[kMoeMaxExperts + 1], before[kMoeMaxExperts], total[kMoeMaxExperts];
    __shared__ uint32_t sums[2][kMoeMaxExperts / 2];       // [0: the rows before, 1: all][16-bit pairs]
    __shared__ int32_t chosen[kRouteTokens * kMoeMaxK];
    __shared__ int32_t part[16];
    const int t = threadIdx.x, lane = t & 63;
    const int row = byte_row(p.E), pieces = row / 16;
    int width = 1;                               // threads a row: a power of two up to 64
    while (width < pieces) width *= 2;
    const uint8_t *counts = reinterpret_cast<const uint8_t *>(p.counts);
    const int piece = t & (width - 1), group = t / width, groups = 1024 / width;
    // (64 tokens have at most 1024 pairs: one a thread)
    const int64_t t0 = (int64_t)blockIdx.x * tokens;
    const int64_t p0 = t0 * p.k, p1 = (t0 + tokens < p.T ? t0 + tokens : p.T) * p.k;
    const int expert = p0 + t < p1 ? p.experts[p0 + t] : -1;
    for (int e = t; e < kMoeMaxExperts; e += 1024) {
        mask[e] = 0;
        if (e < kMoeMaxExperts / 2) sums[0][e] = sums[1][e] = 0;
    }
    uint32_t mine[8] = {}, all[8] = {};          // (at most 16 rows a thread: sums of 1024)
    if (piece < pieces) {
#pragma unroll 4
        for (int r = group; r < nb; r += groups) {
            const u32x4 v = *reinterpret_cast<const u32x4 *>(counts + r * row + 16 * piece);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t even = v[i] & 0x00FF00FFu, odd = (v[i] >> 8) & 0x00FF00FFu;
                all[2 * i] += even;
                all[2 * i + 1] += odd;
                mine[2 * i] += r < (int)blockIdx.x ? even : 0;
                mine[2 * i + 1] += r < (int)blockIdx.x ? odd : 0;
            }
        }
    }
    for (int d = width; d < 64; d *= 2) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            all[i] += (uint32_t)__shfl_xor((int)all[i], d);
            mine[i] += (uint32_t)__shfl_xor((int)mine[i], d);
        }
    }
    __syncthreads();
    if (lane < width && piece < pieces) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            // word i of a piece: experts 4 (i / 2) + i % 2 and two further on
            atomicAdd(&sums[0][8 * piece + i], mine[i]);
            atomicAdd(&sums[1][8 * piece + i], all[i]);
        }
    }
    __syncthreads();
    for (int e = t; e < p.E; e += 1024) {
        const int w = 8 * (e / 16) + 2 * (e % 16 / 4) + (e & 1), up = (e & 2) * 8;
        before[e] = (int)(sums[0][w] >> up & 0xFFFF);
        total[e] = (int)(sums[1][w] >> up & 0xFFFF);
    }
    static_assert(kRouteTokens * kMoeMaxK <= 1024, "a pair a thread");
    if (p0 + t < p1) chosen[t] = expert;
    if (expert >= 0) atomicOr(reinterpret_cast<unsigned long long *>(&mask[expert]), 1ull << (t / p.k));
    __syncthreads();
    scan_experts(total, p.E, base, part);        // (ends with a barrier)
    if (blockIdx.x == 0)
        for (int e = t; e <= p.E; e += 1024) p.offsets[e] = base[e];
    place(p, t0, p0, p1, mask, base, before, chosen);
}

// dlogits = p (u - sum p u): p the softmax over all experts, or over the
// chosen ones (renorm), u the weights' gradients (times `factor`) at the chosen experts and 0
// elsewhere.  16 lanes a token, as in route_select; lane j has the j-th
// choice, and the chosen experts' gradients reach the lanes that hold those
// experts through a row of E floats in LDS (zeroed, written and read by the
// token's own lanes of one wave, with a handover between).
template <int VPL, int C, bool BF16>
__global__ __launch_bounds__(kThreads) void route_bwd(const void *logits, int64_t T, int E, int k, int renorm, float factor,
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
            u = dweights[tok * k + l] * factor;
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

// The gradient through sigmoid scores, at the chosen experts alone:
//
//     renorm:  w_j (u_j - sum_i w_i u_i) (1 - s_j)      w the weights, of sum 1
//     else:    u_j s_j (1 - s_j)
//
// with u the weights' gradients times `factor`.  Only the chosen logits are
// read; a token's row of zeros and k values goes out through LDS.  (16384 tokens, 6 of 160
// experts, bf16: 4.1 us, two trips to memory one after the other, the choice and its logits.)
template <int VPL, int C, bool BF16>
__global__ __launch_bounds__(kThreads) void route_sigmoid_bwd(const void *logits, int64_t T, int E, int k, int renorm,
                                                              float factor, const int32_t *experts, const float *dweights,
                                                              void *dlogits)
{
    __shared__ __attribute__((aligned(16))) float at_chosen[kThreads / kLanes][16 * VPL];
    const int l = threadIdx.x & (kLanes - 1);
    const int64_t tok = (int64_t)blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes;
    if (tok >= T) return;                        // (uniform in the token's 16 lanes)
    float *row = at_chosen[threadIdx.x / kLanes];
    int e = -1;
    float u = 0.0f, x = -INFINITY;
    if (l < k) {
        e = experts[tok * k + l];
        e = e < E ? e : -1;
        if (e >= 0) {
            u = dweights[tok * k + l] * factor;
            const int64_t at = tok * E + e;
            if constexpr (BF16)
                x = open_logit(__builtin_bit_cast(float, (uint32_t) reinterpret_cast<const uint16_t *>(logits)[at] << 16));
            else
                x = open_logit(reinterpret_cast<const float *>(logits)[at]);
        }
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) row[expert_of<C>(i, l)] = 0.0f;
    wave_handover();
    // (1 - s = e^-x / (1 + e^-x); an expert closed since then has no gradient)
    const bool open = x > -INFINITY;
    const float low = expf(-fabsf(x)), half = 1.0f / (1.0f + low);
    const float rest = x >= 0.0f ? low * half : half;
    float d;
    if (renorm) {
        const float from = row_max(fminf(x, 0.0f));
        const float s = open ? expf(fminf(x, 0.0f) - from) * half : 0.0f;
        const float total = row_sum(s), w = open ? s / total : 0.0f;
        d = w * (u - row_sum(w * u)) * rest;
    } else {
        d = u * (x >= 0.0f ? half : low * half) * rest;
    }
    if (e >= 0) row[e] = open ? d : 0.0f;
    wave_handover();
#pragma unroll
    for (int i = 0; i < VPL; i += C) {
        const int first = expert_of<C>(i, l);
        if (first >= E) continue;
        const int64_t at = tok * E + first;
        if constexpr (BF16) {
            __bf16 w[C];
#pragma unroll
            for (int c = 0; c < C; ++c) w[c] = (__bf16)row[first + c];
            __builtin_memcpy(reinterpret_cast<__bf16 *>(dlogits) + at, w, sizeof(w));
        } else {
            float w[C];
#pragma unroll
            for (int c = 0; c < C; ++c) w[c] = row[first + c];
            __builtin_memcpy(reinterpret_cast<float *>(dlogits) + at, w, sizeof(w));
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

// The order of the pairs behind the selecting kernel's counts.
static hipError_t launch_place(const MoeRoute &p, int64_t nb, hipStream_t stream)
{
    if (nb <= kDirect) {
        hipLaunchKernelGGL((route_place<true>), dim3(nb), dim3(kThreads), 0, stream, p, nb);
        return hipGetLastError();
    }
    hipLaunchKernelGGL(route_columns, dim3((p.E + 15) / 16), dim3(1024), 0, stream, p.counts, nb, p.E);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((route_place<false>), dim3(nb), dim3(kThreads), 0, stream, p, nb);
    return hipGetLastError();
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
    return launch_place(p, nb, stream);
}

// A lane's experts: at most 64 of a group's, in whole loads of four where every
// group's logits are whole ones.
int moe_route_grouped_lane(int64_t E, int64_t groups, bool fours)
{
    int runs = 1;
    while (runs < groups) runs *= 2;
    const int64_t lanes = kLanes / runs, per = E / groups;
    int64_t q = (per + lanes - 1) / lanes;
    if (fours) q = (q + 3) / 4 * 4;
    return (int)q;
}

// Tokens a workgroup of T: 16, or 32, while there are no more of them than kBytes, else 64
static int grouped_tokens(int64_t T)
{
    return T <= kRouteTokens ? kRouteTokens : T <= 16 * kBytes ? 16 : T <= 32 * kBytes ? 32 : 64;
}

int64_t moe_route_grouped_workspace_bytes(int64_t T, int64_t E)
{
    const int64_t tokens = grouped_tokens(T), nb = (T + tokens - 1) / tokens;
    if (T <= kRouteTokens) return 0;
    return nb <= kBytes ? nb * byte_row((int)E) : moe_route_workspace_bytes(T, E);
}

hipError_t launch_moe_route_grouped(MoeRouteGrouped g, hipStream_t stream)
{
    const MoeRoute &p = g.r;
    g.tokens = grouped_tokens(p.T);
    const int64_t nb = (p.T + g.tokens - 1) / g.tokens;
    const bool one = p.T <= kRouteTokens;
    const bool fours = p.E / g.groups % 4 == 0 &&
                       ((reinterpret_cast<uintptr_t>(p.logits) | reinterpret_cast<uintptr_t>(g.bias)) & 15) == 0;
    int runs = 1;
    while (runs < g.groups) runs *= 2;
    g.lanes = kLanes / runs;
    g.q = moe_route_grouped_lane(p.E, g.groups, fours);
    g.bytes = !one && nb <= kBytes;
    const bool few = one ? p.T <= 16 : g.tokens == 16;
    auto go = [&](auto vpl, auto c, auto bf16, auto whole) {
        constexpr int V = decltype(vpl)::value, C = decltype(c)::value, MANY = V > 16 ? 512 : 1024;
        constexpr bool B = decltype(bf16)::value, ONE = decltype(whole)::value;
        if (few) hipLaunchKernelGGL((route_choose<V, C, B, ONE, 256>), dim3(nb), dim3(256), 0, stream, g);
        else hipLaunchKernelGGL((route_choose<V, C, B, ONE, MANY>), dim3(nb), dim3(MANY), 0, stream, g);
        return hipGetLastError();
    };
    auto by_type = [&](auto vpl, auto c) {
        if (one) return p.bf16 ? go(vpl, c, std::true_type{}, std::true_type{}) : go(vpl, c, std::false_type{}, std::true_type{});
        return p.bf16 ? go(vpl, c, std::true_type{}, std::false_type{}) : go(vpl, c, std::false_type{}, std::false_type{});
    };
    auto by_load = [&](auto vpl) {
        return fours ? by_type(vpl, std::integral_constant<int, 4>{}) : by_type(vpl, std::integral_constant<int, 1>{});
    };
    hipError_t e;
    if (g.q <= 4) e = by_load(std::integral_constant<int, 4>{});
    else if (g.q <= 8) e = by_load(std::integral_constant<int, 8>{});
    else if (g.q <= 16) e = by_load(std::integral_constant<int, 16>{});
    else if (g.q <= 32) e = by_load(std::integral_constant<int, 32>{});
    else e = by_load(std::integral_constant<int, 64>{});
    if (e != hipSuccess || one) return e;
    if (!g.bytes) return launch_place(p, nb, stream);
    hipLaunchKernelGGL(route_place_bytes, dim3(nb), dim3(1024), 0, stream, p, (int)nb, g.tokens);
    return hipGetLastError();
}

hipError_t launch_moe_route_bwd(const void *logits, int bf16, int64_t T, int E, int k, int sigmoid, int renorm, float factor,
                                const int32_t *experts, const float *dweights, void *dlogits, hipStream_t stream)
{
    const dim3 grid((T + kThreads / kLanes - 1) / (kThreads / kLanes));
    return by_experts(E, logits, dlogits, [&](auto vpl, auto c) {
        constexpr int V = decltype(vpl)::value, C = decltype(c)::value;
        auto go = [&](auto *kernel) {
            hipLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, stream, logits, T, E, k, renorm, factor, experts, dweights,
                               dlogits);
            return hipGetLastError();
        };
        if (sigmoid) return bf16 ? go(&route_sigmoid_bwd<V, C, true>) : go(&route_sigmoid_bwd<V, C, false>);
        return bf16 ? go(&route_bwd<V, C, true>) : go(&route_bwd<V, C, false>);
    });
}

}  // namespace dbs
