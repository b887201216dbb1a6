// moe_core.h -- what the experts' products in bf16 (moe_gemm.hip) and in 8-bit
// integers (i8_gemm.hip) share on the device: the written-out direct-to-LDS
// loads, the tables of groups, and the 256 x 256 core over stages of 128 bytes a
// row.
#pragma once

#include "gemm_kernel.h"
#include "moe.h"
#include "moe_device.h"
#include "moe_tiles.h"

namespace dbs {
namespace {

// Results are stored through the caches: a wave's pieces are half lines, which
// L2 puts together (32768 x 2048 results over 32 experts: 451 us with
// streaming stores, 413 without, in even groups).
constexpr int kStoreCached = 0;
constexpr uint32_t kRowOOB = 0xFF000000u;        // + a row's bytes (at most 2^22) still lies past every resource

// Buffer descriptor (see make_rsrc) as the four words an instruction takes;
// base and bytes are the same in every lane.
__device__ __forceinline__ i32x4 words_of(const void *base, uint32_t bytes)
{
    const uint64_t b = (uint64_t)base;
    return i32x4{__builtin_amdgcn_readfirstlane((int)(uint32_t)b),
                 __builtin_amdgcn_readfirstlane((int)((uint32_t)(b >> 32) & 0xFFFFu)),
                 __builtin_amdgcn_readfirstlane((int)bytes), 0x00020000};
}

// Direct-to-LDS load of BYTES per lane, as lds_dma in gemm_kernel.h, but
// written out: the compiler follows the builtin's loads and waits for all of
// them before any LDS read, which would end the overlap this file's kernels
// are built on.  They wait by count themselves, at every barrier.  Lane i's
// bytes land at lds + dst + BYTES i; nothing is returned to registers.  M0 holds
// the destination; the compiler learns that it is written as an output.
// A descriptor's words come from v_readfirstlane or, respilled, v_readlane, and
// a vector load may read an SGPR that a vector instruction wrote only five wait
// states later (M0 one after it is set).  The compiler does not count them for
// a load inside asm, so they stand here: one move and four of s_nop 3.
template <int BYTES>
__device__ __forceinline__ void dma(const i32x4 &words, uint8_t *lds, uint32_t dst, uint32_t voff)
{
    static_assert(BYTES == 4 || BYTES == 16, "dword or dwordx4");
#if DBS_LDS_POISON
    const uint32_t lane = __builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u));
    if constexpr (BYTES == 4)
        *reinterpret_cast<uint32_t *>(lds + dst + 4 * lane) = ~0u;
    else
        *reinterpret_cast<i32x4 *>(lds + dst + 16 * lane) = i32x4{-1, -1, -1, -1};
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#endif
    const uint32_t to = (uint32_t)(uintptr_t)(lds_void *)lds + dst;
    uint32_t m0;
    if constexpr (BYTES == 4)
        asm volatile("s_mov_b32 m0, %1\n\ts_nop 3\n\tbuffer_load_dword %2, %3, 0 offen lds"
                     : "=&{m0}"(m0)
                     : "s"(to), "v"(voff), "s"(words)
                     : "memory");
    else
        asm volatile("s_mov_b32 m0, %1\n\ts_nop 3\n\tbuffer_load_dwordx4 %2, %3, 0 offen lds"
                     : "=&{m0}"(m0)
                     : "s"(to), "v"(voff), "s"(words)
                     : "memory");
}

// Two wave-loads to neighbouring KiB, or four, the second two `apart` bytes
// behind the first, from one descriptor, at offsets max(x, y) -- y is 0 or, where
// a lane has nothing to load, an offset out of bounds -- or, with SUM, x + y, y
// the same in every lane.  The arithmetic stands in the descriptor's wait
// states; a vector instruction may read an SGPR two states after one wrote it.
// 32 experts of 4096 x 2048, 32768 rows, MN-major: 519 us, 532 with the loads
// one by one and s_nop 3 before each.
#define DBS_LOAD_PAIR(OP, Y)                                                                                   \
    asm volatile("s_mov_b32 m0, %3\n\ts_nop 0\n\t"                                                            \
                 OP " %1, %6, %4\n\t"                                                                          \
                 OP " %2, %7, %5\n\t"                                                                          \
                 "s_nop 0\n\t"                                                                                 \
                 "buffer_load_dwordx4 %1, %8, 0 offen lds\n\t"                                                 \
                 "s_add_u32 m0, m0, 0x400\n\ts_nop 0\n\t"                                                     \
                 "buffer_load_dwordx4 %2, %8, 0 offen lds"                                                     \
                 : "=&{m0}"(m0), "=&v"(off[0]), "=&v"(off[1])                                                  \
                 : "s"(to), "v"(x[0]), "v"(x[1]), Y(y[0]), Y(y[1]), "s"(words)                                 \
                 : "memory", "scc")
#define DBS_LOAD_FOUR(FIRST, OP, Y)                                                                            \
    asm volatile("s_mov_b32 m0, %5\n\t" FIRST                                                                  \
                 OP " %1, %10, %6\n\t"                                                                         \
                 OP " %2, %11, %7\n\t"                                                                         \
                 OP " %3, %12, %8\n\t"                                                                         \
                 OP " %4, %13, %9\n\t"                                                                         \
                 "buffer_load_dwordx4 %1, %14, 0 offen lds\n\t"                                                \
                 "s_add_u32 m0, m0, 0x400\n\ts_nop 0\n\t"                                                     \
                 "buffer_load_dwordx4 %2, %14, 0 offen lds\n\t"                                                \
                 "s_add_u32 m0, m0, %15\n\ts_nop 0\n\t"                                                       \
                 "buffer_load_dwordx4 %3, %14, 0 offen lds\n\t"                                                \
                 "s_add_u32 m0, m0, 0x400\n\ts_nop 0\n\t"                                                     \
                 "buffer_load_dwordx4 %4, %14, 0 offen lds"                                                    \
                 : "=&{m0}"(m0), "=&v"(off[0]), "=&v"(off[1]), "=&v"(off[2]), "=&v"(off[3])                    \
                 : "s"(to), "v"(x[0]), "v"(x[1]), "v"(x[2]), "v"(x[3]), Y(y[0]), Y(y[1]), Y(y[2]), Y(y[3]),    \
                   "s"(words), "s"(apart - 1024)                                                               \
                 : "memory", "scc")

template <bool SUM, int N>
__device__ __forceinline__ void dma_group(const i32x4 &words, uint8_t *lds, uint32_t dst, const uint32_t (&x)[N],
                                          const uint32_t (&y)[N], uint32_t apart = 0)
{
    static_assert(N == 2 || N == 4, "one pair or two");
#if DBS_LDS_POISON
#pragma unroll
    for (int i = 0; i < N; ++i)
        dma<16>(words, lds, dst + (i & 1) * 1024 + (i >> 1) * apart, SUM ? x[i] + y[i] : max(x[i], y[i]));
#else
    const uint32_t to = (uint32_t)(uintptr_t)(lds_void *)lds + dst;
    uint32_t m0, off[N];
    if constexpr (N == 2 && SUM) DBS_LOAD_PAIR("v_add_u32", "s");
    else if constexpr (N == 2) DBS_LOAD_PAIR("v_max_u32", "v");
    else if constexpr (SUM) DBS_LOAD_FOUR("s_nop 0\n\t", "v_add_u32", "s");
    else DBS_LOAD_FOUR("", "v_max_u32", "v");
#endif
}

struct Lane {
    int lane, h, lr, w, wm, wn;
};

__device__ __forceinline__ Lane lane_of()
{
    Lane c;
    c.lane = threadIdx.x & 63;
    c.h = c.lane >> 5;
    c.lr = c.lane & 31;
    c.w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    c.wm = c.w / 4;
    c.wn = c.w % 4;
    return c;
}

// ------------------------------------------------------------ group tables

// first[g] = first row of group g (g <= E; offsets clamped to 0 .. M and made
// ascending; with FIRST), and at[g] = units of work before group g, per(rows)
// of them in a group: by one wave, the others wait at the caller's barrier.
// A lane has ceil(E / 64) groups in a row, so that all loads are under way
// together (1024 experts: 16 trips to memory one after the other before).
template <bool FIRST, class T, class PER>
__device__ __forceinline__ void group_table(int32_t *first, T *at, const int32_t *offsets, int E, int M, const Lane &c,
                                            PER &&per)
{
    constexpr int kMost = kMoeMaxExperts / 64;
    const int S = (E + 63) / 64, g0 = c.lane * S;
    int end[kMost];
#pragma unroll
    for (int i = 0; i < kMost; ++i) {
        if (i == S) break;
        end[i] = offsets[min(g0 + i + 1, E)];
    }
    const int start = min(max(offsets[0], 0), M);
    int top = start;
#pragma unroll
    for (int i = 0; i < kMost; ++i) {
        if (i == S) break;
        end[i] = min(max(end[i], 0), M);
        top = max(top, end[i]);
    }
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int o = __shfl_up(top, d);
        if (c.lane >= d) top = max(top, o);
    }
    int lo = __shfl_up(top, 1);                // the lane's first row
    lo = c.lane == 0 ? start : lo;
    int sum = 0, row = lo;
#pragma unroll
    for (int i = 0; i < kMost; ++i) {
        if (i == S) break;
        end[i] = max(end[i], row);
        sum += g0 + i < E ? per(end[i] - row) : 0;
        row = end[i];
    }
    int work = sum;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int o = __shfl_up(work, d);
        if (c.lane >= d) work += o;
    }
    work -= sum;
    row = lo;
#pragma unroll
    for (int i = 0; i < kMost; ++i) {
        if (i == S) break;
        if (g0 + i < E) {
            if constexpr (FIRST) first[g0 + i] = row;
            at[g0 + i] = (T)work;
            work += per(end[i] - row);
            row = end[i];
            if (g0 + i == E - 1) {
                if constexpr (FIRST) first[E] = row;
                at[E] = (T)work;
            }
        }
    }
}

// The last group g with at[g] <= id (groups without work have equal
// neighbours): every ceil(E / 64)-th entry, then those behind the last of them.
template <class T>
__device__ __forceinline__ int group_of(const T *at, int E, int id, const Lane &c)
{
    const int S = (E + 63) / 64;
    int g = c.lane * S;
    const int block = __builtin_amdgcn_readfirstlane((__popcll(__ballot(g < E && (int)at[min(g, E)] <= id)) - 1) * S);
    if (S == 1) return block;
    g = block + c.lane;
    return block + __builtin_amdgcn_readfirstlane(__popcll(__ballot(c.lane < S && g < E && (int)at[min(g, E)] <= id)) - 1);
}

__device__ __forceinline__ int first_tile()
{
    // workgroup w runs on XCD w % 8: every XCD takes a run of tiles
    const int nwg = gridDim.x, wg = blockIdx.x;
    return (nwg & 7) == 0 ? (wg & 7) * (nwg >> 3) + (wg >> 3) : wg;
}

// --------------------------------------------------- the 256 x 256 x 64 core

// 256 x 256 output tiles over stages of 64, 8 waves (2 x 4, two per SIMD),
// each owning 128 x 64.  A stage is four parts of 16 KiB -- A's rows (or
// columns) 0 .. 127 and 128 .. 255, B's likewise -- in one of two LDS slots,
// and is computed in two turns of 32 MFMAs a wave.  A wave reads the parts of
// a turn whole into registers, so their places in the slot are free again at
// once, and their refill for the stage after next starts a turn later: loads
// get at least two turns of the four that two stages take to land, with two
// slots.  (Rows that nothing else has touched come from HBM: with loads of one
// stage's lead, waited for in full at its end, the same tiles took a quarter
// longer.)
//
// The two waves of a SIMD take turns: while one reads its parts and issues
// its loads, the other runs its MFMAs, a workgroup barrier between.  Waves
// 4 .. 7 start one turn late.
//
//   turn   reads                  loads issued                      MFMAs
//   0      A lo, B lo, B hi       A hi of stage s + 1               A lo (B lo, B hi)
//   1      A hi                   A lo, B lo, B hi of stage s + 2   A hi (B hi, B lo)
//
// At the end of a turn's reads a wave waits for its loads of the parts read in
// the turn after: the newer kInFlight wave-loads may be under way by then (the
// turn's own and one turn's before it: 2 + 6).  Its own reads are complete
// before the barrier that lets others refill their place.
//
// What bounds it is the clock that the power leaves and, close behind, the
// 64 KiB a stage that come into LDS: 32768 rows over 32 experts, 4096 x 2048,
// in even groups take 431 us (1.28 PFLOP/s), on zeros 343.  A tile costs 1.5 us
// a stage and 6 us of storing, in which all CUs write at once.
constexpr int kPart = 128 * kRowBytes, kSlot = 4 * kPart, kInFlight = 8;
enum PartId : int { kALo = 0, kAHi = 1, kBLo = 2, kBHi = 3 };
constexpr int kStage = 2 * kSlot;              // LDS offset of the waves' output buffers, 2 KiB each
constexpr int kCoreLds = kStage + 8 * 2048;

// K-major part: 128 rows of 128 bytes, chunks swizzled as everywhere (swz);
// wave-load L (0 .. 15) covers rows 8 L .. 8 L + 7.  MN-major part: 64 K-rows
// of 128 columns (256 bytes), wave-load L covers K-rows 4 L .. 4 L + 3.  Wave
// w issues wave-loads 2 w and 2 w + 1.
//
// The math is v_mfma_f32_16x16x32_bf16: the products of even groups ran at 1.30
// PFLOP/s with it and at 1.22 with 32x32x16, both bound by the clock that
// power leaves (an accumulator is read and written half as often).  Its
// lane l holds row (or column) l % 16 and eight K of a 16 x 32 operand block,
// and of the result, with B's block as the first operand, row l % 16 of A's
// and columns 4 (l / 16) .. + 3 of B's.  The lane's K are 8 kgroup(l / 16) ..,
// the same order for A and B: one LDS pass of 16-byte reads takes lanes of
// groups 0 and 2 (or 1 and 3) together, which then read neighbouring chunks
// of their rows, apart under the swizzle (chunks two apart were not: half of
// the LDS cycles were conflicts).
constexpr int kMnRow = 256;
typedef __attribute__((ext_vector_type(4))) float f32x4;

// The lane's byte offset in wave-loads 2 w and 2 w + 1 of an MN-major part
// whose K-rows lie ld bytes apart in memory (8 w .. 8 w + 7 share the bits above 2).
__device__ __forceinline__ uint32_t mn_part_lane(const Lane &c, int ld)
{
    const int r = c.lane >> 4;
    return (uint32_t)(r * ld + (((c.lane & 15) ^ mn_swz(8 * c.w + r)) << 4));
}

// The lane's address of operand block 0, k-step 0 of a part: rows (columns)
// 32 block0 .. + 15.
template <bool MN>
__device__ __forceinline__ uint32_t part_base(const Lane &c, int block0)
{
    const int j = c.lane & 15, g = c.lane >> 4;
    if constexpr (MN) {
        // transposed reads: lane j of a group addresses K-row j / 4 of four at columns 4 (j % 4) ..
        const int r = 8 * kgroup(g) + (j >> 2);
        return (uint32_t)(r * kMnRow + ((64 * block0 + 8 * (j & 3)) ^ (mn_swz(r) << 4)));
    } else {
        const int r = 32 * block0 + j;
        return (uint32_t)(r * kRowBytes + ((kgroup(g) ^ swz(r)) << 4));
    }
}

// k-step kk (32 of the summed axis) of rows (columns) 64 i + 16 u .. + 15 from
// the lane's base on
template <bool MN>
__device__ __forceinline__ bf16x8 part_frag(const uint8_t *lds, uint32_t base, int kk, int i, int u)
{
    if constexpr (MN) {
        typedef __attribute__((address_space(3))) i16x4 lds_i16x4;
        const uint8_t *x = lds + (base ^ (uint32_t)(128 * i + 32 * u)) + kk * 32 * kMnRow;
        const i32x2 lo = __builtin_bit_cast(i32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4 *)x));
        const i32x2 hi = __builtin_bit_cast(i32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4 *)(x + 4 * kMnRow)));
        return __builtin_bit_cast(bf16x8, i32x4{lo[0], lo[1], hi[0], hi[1]});
    } else {
        // (16 rows further down bit 1 of the swizzle changes)
        return lds_read<bf16x8>(lds, (base ^ (uint32_t)((kk << 6) ^ (u << 5))) + (uint32_t)((64 * i + 16 * u) * kRowBytes));
    }
}

template <int N>
__device__ __forceinline__ void turn_end()
{
    DBS_FENCE();
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"i"(N) : "memory");
    DBS_FENCE();
}

__device__ __forceinline__ void turn_end_math()
{
    DBS_FENCE();
    __builtin_amdgcn_s_setprio(0);
    asm volatile("s_barrier" ::: "memory");
    DBS_FENCE();
}

// The arithmetic of a kernel: four results a lane of a 16 x 16 block from 64 bytes
// of 16 rows (columns) of each operand, of which lane l holds 16.
struct MulBf16 {
    typedef f32x4 Sum;
    static __device__ __forceinline__ f32x4 mul(bf16x8 b, bf16x8 a, f32x4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(b, a, c, 0, 0, 0);
    }
};

// A wave's results: 16 x 16 blocks [rows 64 (i / 4) + 32 (i / 2 % 2) .. of the
// wave's 128, 16 (i % 2) further down][columns 16 (j % 2) of part j / 2].
template <class MUL>
using Acc = typename MUL::Sum[8][4];

template <bool BMN>
__device__ __forceinline__ void read_b(bf16x8 (&b)[4], const uint8_t *lds, uint32_t base)
{
#pragma unroll
    for (int kk = 0; kk < 2; ++kk)
#pragma unroll
        for (int u = 0; u < 2; ++u) b[2 * kk + u] = part_frag<BMN>(lds, base, kk, 0, u);
}

// One stage out of slot `slot`.  NLO, NHI: blocks per wave in the two halves
// of A (fewer than 2 where a group ends).  advance() moves the loads on to the
// next stage, load(part, slot) issues the two wave-loads of a part of A, or
// (kBLo) the four of both parts of B.
// extra: STORES stores of the last tile's results went out between the loads
// awaited here and now, and may still be under way.
template <class MUL, bool AMN, bool BMN, int NLO, int NHI, class LOAD, class ADVANCE, int STORES>
__device__ __forceinline__ void core_stage(Acc<MUL> &acc, const uint8_t *lds, uint32_t fa, uint32_t fb, int slot, int extra,
                                           LOAD &&load, ADVANCE &&advance, std::integral_constant<int, STORES>)
{
    bf16x8 a[4][2], b0[4], b1[4];          // b: [2 kk + u]
    const uint32_t so = (uint32_t)(slot * kSlot);
    auto wait = [&] {
        if (extra) turn_end<kInFlight + STORES>();
        else turn_end<kInFlight>();
    };
    auto read_a = [&](int part, int n) {
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
#pragma unroll
            for (int i = 0; i < 2 * n; ++i) a[i][kk] = part_frag<AMN>(lds, fa + so + part * kPart, kk, i >> 1, i & 1);
    };
    auto math = [&](int half, int j, int n, const bf16x8 (&b)[4]) {
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
#pragma unroll
            for (int i = 0; i < 2 * n; ++i)
#pragma unroll
                for (int u = 0; u < 2; ++u)
                    acc[4 * half + i][2 * j + u] = MUL::mul(b[2 * kk + u], a[i][kk], acc[4 * half + i][2 * j + u]);
    };
    // turn 0
    read_a(kALo, NLO);
    read_b<BMN>(b0, lds, fb + so + kBLo * kPart);
    read_b<BMN>(b1, lds, fb + so + kBHi * kPart);
    load(kAHi, slot ^ 1);
    wait();
    __builtin_amdgcn_s_setprio(1);
    math(0, 0, NLO, b0);
    math(0, 1, NLO, b1);
    turn_end_math();
    // turn 1
    read_a(kAHi, NHI);
    advance();
    load(kALo, slot);
    load(kBLo, slot);
    wait();
    __builtin_amdgcn_s_setprio(1);
    math(1, 1, NHI, b1);
    math(1, 0, NHI, b0);
    turn_end_math();
}

// One 32 x 32 block of results as bf16 rows r0 .. mend-1, columns n0 ..
// ncols-1 of D (ld columns), through the wave's 2 KiB buffer and in 16-byte
// pieces (vec) or by element; value(u, v, q): register q of 16 x 16 block (u, v).
// Neighbouring lanes then write neighbouring pieces of a row: exchanged
// between lanes instead (v_permlane16_swap), with 16 rows to the 16 lanes next to
// each other, dW of 32 experts took 564 us where this takes 541.
template <class VALUE>
__device__ __forceinline__ void store_block(uint8_t *buf, uint8_t *D, int64_t ld, int r0, int mend, int n0, int ncols,
                                            int vec, Lane c, VALUE &&value)
{
    // (addresses are made here, not before the tile's stages, whose registers they would take)
    asm volatile("" : "+v"(c.lane));
    const int left = __builtin_amdgcn_readfirstlane(max(0, min(32, mend - r0)));
    const __amdgpu_buffer_rsrc_t rd = make_rsrc(D + (int64_t)r0 * ld * 2, (uint32_t)left * (uint32_t)ld * 2u);
    // block g's four values of consecutive columns lie at row and column
    const int row0 = c.lane & 15, col0 = 4 * (c.lane >> 4);
    if (vec) {
        wave_handover();                     // (the block before has been read)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const int u = g >> 1, v = g & 1, row = 16 * u + row0, col = 16 * v + col0;
            *reinterpret_cast<u32x2 *>(buf + row * 64 + (((col >> 3) ^ ((row >> 1) & 3)) << 4) + 2 * (col & 4)) =
                u32x2{pack_bf16(value(u, v, 0), value(u, v, 1)), pack_bf16(value(u, v, 2), value(u, v, 3))};
        }
        wave_handover();
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int r = q * 16 + (c.lane >> 2), ch = c.lane & 3, n = n0 + ch * 8;
            const i32x4 v = *reinterpret_cast<const i32x4 *>(buf + r * 64 + 16 * (ch ^ ((r >> 1) & 3)));
            __builtin_amdgcn_raw_buffer_store_b128(v, rd, n < ncols ? (uint32_t)(r * (int)ld + n) * 2u : kOOB, 0,
                                                   kStoreCached);
        }
    } else {
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const int u = g >> 1, v = g & 1;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int n = n0 + 16 * v + col0 + q;
                __builtin_amdgcn_raw_buffer_store_b16((uint16_t)pack_bf16(value(u, v, q), 0.0f), rd,
                                                      n < ncols ? (uint32_t)((16 * u + row0) * (int)ld + n) * 2u : kOOB, 0,
                                                      kStoreCached);
            }
        }
    }
}

}  // namespace
}  // namespace dbs
