// moe_gemm.hip -- gfx950 kernels of the experts' products (bf16, fp32 sums):
//
//   tiles   D[i, n]      = sum_k X[rows[i], k] W_g[n, k]      i in group g; W_g K-major (N x K)
//           D[i, n]      = sum_k X[rows[i], k] W_g[k, n]      W_g MN-major (K x N): the rows' gradient
//           D[i, f]      = silu(h[f]) h[F + f]                h = the first form's row, F = N / 2 (the gate)
//   dw      dW_g[n, k]   = sum_i dY[i, n] X[rows[i], k]       over the rows i of group g
//
// The groups' row offsets are read on the device: a workgroup turns them
// into a table of first tiles in LDS, so a router's output needs no copy to
// the host.  Many rows per expert are bound by the matrix cores (256 x 256
// tiles: 1.3 PFLOP/s), few by the reading of W (64-row tiles: up to 5.8 TB/s).
//
// * Rows.  A gathered row's byte offset is taken from `rows` once per output
//   tile and lives in one register per wave-load, so gathering costs one add
//   per load and stage; the sorted copy of X that it replaces would cost a
//   write and a read of M x K.  Offsets are 32 bits from one buffer
//   resource: a gathered X stays below kRowOOB bytes.
// * Bounds.  Offsets are clamped to 0 .. M and made ascending, row indices
//   outside X read zero rows, and every resource ends with its operand: no
//   value in device memory leads outside the caller's tensors.
// * The gate.  A tile's 256 rows of W are 128 of the gate matrix and the 128
//   of the up matrix that meet them, alternating by 32, so one lane holds
//   both factors of an output and h never leaves the registers.
// * dw.  The summed axis is the group's rows: both operands are MN-major
//   (transposed LDS reads), the number of stages differs from tile to tile,
//   and the resources of a stage's rows end with the group, so rows past it
//   read zero in both factors.  An expert without rows gets zeros (or, when
//   accumulating, nothing).
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

// A wave's results: 16 x 16 blocks [rows 64 (i / 4) + 32 (i / 2 % 2) .. of the
// wave's 128, 16 (i % 2) further down][columns 16 (j % 2) of part j / 2].
typedef f32x4 Acc[8][4];

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
template <bool AMN, bool BMN, int NLO, int NHI, class LOAD, class ADVANCE, int STORES>
__device__ __forceinline__ void core_stage(Acc &acc, const uint8_t *lds, uint32_t fa, uint32_t fb, int slot, int extra,
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
                    acc[4 * half + i][2 * j + u] =
                        __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[2 * kk + u], a[i][kk], acc[4 * half + i][2 * j + u], 0, 0, 0);
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

// ------------------------------------------------------------------- tiles

template <int TM>
__device__ __forceinline__ void fill_table(Table<TM> &tab, const MoeGemm &p, const Lane &c)
{
    if (c.w == 0)
        group_table<true>(tab.first, tab.whole, p.offsets, p.E, p.M, c, [](int rows) { return Table<TM>::whole_of(rows); });
    else if (c.w < TM / 64)
        group_table<false>(tab.first, tab.rest[c.w - 1], p.offsets, p.E, p.M, c,
                           [&](int rows) { return Table<TM>::rest_of(rows, c.w); });
}

// Rows from .. to-1 of D are zero (those before the first group and behind the last).
__device__ __forceinline__ void zero_rows(const MoeGemm &p, int64_t from, int64_t to)
{
    const int64_t bytes = (to - from) * p.ncols * 2;
    uint8_t *z = p.D + from * p.ncols * 2;
    const int64_t me = (int64_t)blockIdx.x * blockDim.x + threadIdx.x, all = (int64_t)gridDim.x * blockDim.x;
    if (p.vec)
        for (int64_t o = me * 16; o < bytes; o += all * 16) *reinterpret_cast<i32x4 *>(z + o) = i32x4{};
    else
        for (int64_t o = me * 2; o < bytes; o += all * 2) *reinterpret_cast<uint16_t *>(z + o) = 0;
}

// 256-row tiles, or of 128 rows (TM) where a call has too few of the large ones
// for the CUs: the same stages, A's upper half filled with zeros and not
// multiplied, 1.1 us in place of 1.3.  BMN: W MN-major; GATE: see the head of the file.
//
// 32768 rows of 32 uneven experts, 4096 x 2048 MN-major: 491 us (1.12
// PFLOP/s): 4.1 tiles' work a CU, of which the busiest have 4.7, with rests
// that cost more than their share; in even groups 431.  24594 rows of 64 very
// uneven experts, 1416 x 2048: 186 us (0.77 PFLOP/s), where groups of 1.5
// tile rows leave a third of the tiles partly empty.
template <int TM, bool BMN, bool GATE>
__global__ __launch_bounds__(512, 1) void moe_tiles(MoeGemm p)
{
    __shared__ __attribute__((aligned(1024))) uint8_t lds[kCoreLds];
    __shared__ Table<TM> tab;
    __shared__ uint32_t rowbuf[256];
    static_assert(!(GATE && BMN), "the gate takes K-major matrices");
    constexpr int TNO = GATE ? 128 : 256;              // output columns of a tile
    constexpr int kStores = GATE ? 8 : 16;             // store instructions of a whole tile (vec)

    Lane c = lane_of();
    const int lda = p.K * 2, ldb = BMN ? p.N * 2 : lda;
    const int tiles_n = (p.ncols + TNO - 1) / TNO;
    fill_table(tab, p, c);
    __syncthreads();
    zero_rows(p, 0, tab.first[0]);
    zero_rows(p, tab.first[p.E], p.M);
    const int ntiles = count_tiles(tab, p.E, tiles_n);
    const int nwg = gridDim.x, self = first_tile();
    if (self >= ntiles) return;
    // at least three stages (the surplus reads zeros): the next tile's row
    // indices land within a tile (see rowbuf)
    const int nk = max((p.K + 63) / 64, 3);
    auto find = [&](int round) {
        return find_tile(tab, p.E, ntiles, tiles_n, TNO, snake(round, nwg, self),
                         [&](const auto *at, int id) { return group_of(at, p.E, id, c); });
    };

    // What the loads read: stage lk of the tile behind ra and rb.
    i32x4 ra, rb;
    uint32_t aoff[4];                     // the lane's row offsets in ra: A lo's two wave-loads, A hi's
    int f0 = 0, lk = 0, first_k = 0;
    uint32_t x4 = (uint32_t)(((c.lane & 7) ^ (c.lane >> 3)) << 4);
    uint32_t lb = BMN ? mn_part_lane(c, ldb) : (uint32_t)((c.lane >> 3) * ldb);
    // Row indices of the tile `r` on their way into rowbuf (lanes past the
    // group's end load zeros, which aim does not use)
    auto fetch = [&](const RowTile &r) {
        const int n = max(r.mend - r.m0, 0);
        const i32x4 rr = words_of(p.rows ? p.rows + r.m0 : nullptr, p.rows ? (uint32_t)min(n, TM) * 4u : 0u);
        dma<4>(rr, reinterpret_cast<uint8_t *>(rowbuf), (c.w & 3) * 256, (uint32_t)((c.w & 3) * 256 + c.lane * 4));
    };
    auto aim = [&](const RowTile &r) {
        // Rows of a K-major W lie 2 K bytes apart: where that is a large power of
        // two, workgroups in step read from few channels of the memory at a time.
        // So the walk along K starts elsewhere for every expert and 2048 columns,
        // which workgroups that share rows in an XCD's L2 have in common (16
        // experts of 4096 x 4096: 64 rows each 128 -> 98 us, 256 rows 143 -> 130
        // us; no difference where W is not what bounds).
        lk = first_k = BMN ? 0 : (r.g * 7 + (r.n0 >> 11) * 5) % nk;
        if (r.blocks == 0) {
            ra = rb = words_of(nullptr, 0);
            return;
        }
        const int64_t wbytes = (int64_t)p.N * p.K * 2;
        const uint8_t *wg = p.W + r.g * wbytes;
        f0 = r.n0;
        if constexpr (BMN)
            rb = words_of(wg + r.n0 * 2, (uint32_t)(wbytes - r.n0 * 2));
        else if constexpr (GATE)
            rb = words_of(wg, (uint32_t)wbytes);
        else
            rb = words_of(wg + (int64_t)r.n0 * lda, (uint32_t)(min(p.N - r.n0, 256) * lda));
        const int left = min(r.mend - r.m0, TM);
        const uint32_t have = p.rows ? (uint32_t)p.T : (uint32_t)left;
        ra = words_of(p.rows ? p.X : p.X + (int64_t)r.m0 * lda, have * (uint32_t)lda);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int m = (q >> 1) * 128 + c.w * 16 + (q & 1) * 8 + (c.lane >> 3);
            const uint32_t row = p.rows ? rowbuf[m] : (uint32_t)m;
            aoff[q] = m < left && row < have ? row * (uint32_t)lda : kRowOOB;
        }
    };
    auto load = [&](int part, int slot) {
        const uint32_t dst = slot * kSlot + part * kPart + c.w * 2048;
        // the lane's bytes of a K-major row, and the least offset they lead to (past the row's end out of bounds)
        uint32_t kc[2], least[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            kc[q] = (x4 ^ (uint32_t)(((c.w * 2 + q) & 7) << 4)) + (uint32_t)(lk * kRowBytes);
            least[q] = kc[q] < (uint32_t)lda ? 0u : kRowOOB;
        }
        if (part == kALo || part == kAHi) {
            const int i = part == kAHi ? 2 : 0;
            dma_group<false, 2>(ra, lds, dst, {aoff[i] + kc[0], aoff[i + 1] + kc[1]}, least);
            return;
        }
        uint32_t x[4], y[4];                   // [2 j + q]: part j of B
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int j = i >> 1, L = c.w * 2 + (i & 1);
            if constexpr (BMN) {
                const uint32_t row = (uint32_t)(lk * 64 + L * 4);          // four K-rows a wave-load
                x[i] = lb + row * (uint32_t)ldb + j * 256;
                y[i] = row < (uint32_t)p.K ? 0u : kOOB;
            } else if constexpr (GATE) {
                const int f = f0 + L * 8;                                  // of matrix j
                x[i] = lb + (uint32_t)(j * p.ncols + f) * (uint32_t)lda + kc[i & 1];
                y[i] = f + (c.lane >> 3) < p.ncols ? least[i & 1] : kOOB;
            } else {
                // wave column L / 4's rows: 32 of its 64
                x[i] = lb + (uint32_t)(((L >> 2) * 64 + j * 32 + (L & 3) * 8) * lda) + kc[i & 1];
                y[i] = least[i & 1];
            }
        }
        dma_group<false, 4>(rb, lds, dst, x, y, kPart);
    };

    RowTile cur = find(0), next = cur;
    auto advance = [&] {
        if (++lk == nk) lk = 0;
        if (lk == first_k) aim(next);
    };
    fetch(cur);
    turn_end<0>();
    aim(cur);
    load(kALo, 0);
    load(kBLo, 0);
    load(kAHi, 0);
    advance();
    load(kALo, 1);
    load(kBLo, 1);
    uint32_t fa = part_base<false>(c, c.wm), fb = part_base<BMN>(c, c.wn);
    uint8_t *buf = lds + kStage + c.w * 2048;
    turn_end<kInFlight>();

    int slot = 0, round = 0, stored = 0;
    auto run = [&](auto nlo, auto nhi) {
        constexpr int NLO = decltype(nlo)::value, NHI = decltype(nhi)::value;
        Acc acc;
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{};
        if (c.w >= 4) asm volatile("s_barrier" ::: "memory");      // one turn behind
#pragma clang loop unroll(disable)
        for (int s = 0; s < nk; ++s) {
            asm volatile("" : "+v"(x4), "+v"(lb), "+v"(fa), "+v"(fb));
            if (s == 0) fetch(next);
            core_stage<false, BMN, NLO, NHI>(
                acc, lds, fa, fb, slot, s == 0 ? stored : 0, load, advance,
                std::integral_constant<int, kStores>{});
            slot ^= 1;
        }
        if (c.w < 4) asm volatile("s_barrier" ::: "memory");
        DBS_FENCE();
#pragma unroll
        for (int i = 0; i < NLO + NHI; ++i) {
            const int r0 = cur.m0 + (2 * i + c.wm) * 32;
            if constexpr (GATE) {
                store_block(buf, p.D, p.ncols, r0, cur.mend, cur.n0 + c.wn * 32, p.ncols, p.vec, c,
                            [&](int u, int v, int q) { return gated(acc[2 * i + u][v][q], acc[2 * i + u][2 + v][q]); });
            } else {
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    store_block(buf, p.D, p.ncols, r0, cur.mend, cur.n0 + (BMN ? j * 128 + c.wn * 32 : c.wn * 64 + j * 32),
                                p.ncols, p.vec, c,
                                      [&](int u, int v, int q) { return acc[2 * i + u][2 * j + v][q]; });
            }
        }
        stored = p.vec && NLO + NHI == 4;
    };
    using I0 = std::integral_constant<int, 0>;
    using I1 = std::integral_constant<int, 1>;
    using I2 = std::integral_constant<int, 2>;
    for (;;) {
        next = find(++round);
        if (TM == 256 && cur.blocks == 4) run(I2{}, std::integral_constant<int, TM == 256 ? 2 : 0>{});
        else if (TM == 256 && cur.blocks == 3) run(I2{}, std::integral_constant<int, TM == 256>{});
        else if (cur.blocks == 2) run(I2{}, I0{});
        else run(I1{}, I0{});
        if (next.blocks == 0) break;
        cur = next;
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // nothing is left to land in LDS
}

// 64-row tiles over a deep ring, for a few rows per expert: the time is the
// reading of W, or a few workgroups' walk along K, where a stage costs the
// loads' latency over the stages they are ahead.  64 columns and eight slots
// of 16 KiB; an MN-major W 128 columns and six slots of 24 KiB (its pieces of
// memory are a tile's K-rows, 256 bytes).  8 waves (4 x 2) of 16 rows and
// half of the columns.  With the gate a wave's 32 rows of W are 16 gate rows
// and the 16 up rows that meet them.
//
// 384 rows on 96 of 128 experts behind the gate, 768 x 4096: 209 us for 1.2 GB
// (5.8 TB/s); one token on 8 experts, 1408 x 2048: 22.6 us for 92 MB (4.1 TB/s:
// 352 tiles on 256 CUs, and the way into the kernel).  Against 64 x 256 tiles over
// three slots (0.7 us a stage): 8 experts of 4096 x 4096, 4 rows 42 us against
// 45, 32 rows 44 against 63; 64 experts of 2816 x 2048, 16 rows 143 against 169.
template <bool BMN>
struct Deep {
    static constexpr int TN = BMN ? 128 : 64, NS = BMN ? 6 : 8, NB = TN / 32, QB = TN / 64;
    static constexpr int kA = 64 * kRowBytes, kSlot = kA + TN * kRowBytes, kWait = (NS - 2) * (1 + QB);
};

template <bool BMN, bool GATE>
__global__ __launch_bounds__(512, 1) void moe_tiles_64(MoeGemm p)
{
    using S = Deep<BMN>;
    constexpr int NB = S::NB;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[S::NS * S::kSlot];
    __shared__ Table<64> tab;
    static_assert(!(GATE && BMN), "the gate takes K-major matrices");
    constexpr int TNO = GATE ? S::TN / 2 : S::TN;

    const Lane c = lane_of();
    const int wm = c.w >> 1, wn = c.w & 1, j = c.lane & 15, g = c.lane >> 4;
    const int lda = p.K * 2, ldb = BMN ? p.N * 2 : lda;
    const int tiles_n = (p.ncols + TNO - 1) / TNO;
    fill_table(tab, p, c);
    __syncthreads();
    zero_rows(p, 0, tab.first[0]);
    zero_rows(p, tab.first[p.E], p.M);
    const int ntiles = count_tiles(tab, p.E, tiles_n);
    const int nwg = gridDim.x;
    int tile = first_tile();
    if (tile >= ntiles) return;
    const int nk = max((p.K + 63) / 64, S::NS - 1);
    auto find = [&](int id) {
        return find_tile(tab, p.E, ntiles, tiles_n, TNO, id,
                         [&](const auto *at, int n) { return group_of(at, p.E, n, c); });
    };

    // wave w loads rows 8 w .. of A and of W (K-rows of an MN-major W)
    i32x4 ra, rb;
    const int lrow = 8 * c.w + (c.lane >> 3);
    int rot = 0;
    uint32_t aoff = 0, boff = BMN ? mn_part_lane(c, ldb) + (uint32_t)(8 * c.w * ldb) : 0u, row = 0;
    uint32_t kx = (uint32_t)(((c.lane & 7) ^ swz(lrow)) << 4);     // the lane's chunk of its row
    auto fetch = [&](const RowTile &r) {
        row = !p.rows ? (uint32_t)lrow : r.m0 + lrow < r.mend ? (uint32_t)p.rows[r.m0 + lrow] : ~0u;
    };
    auto aim = [&](const RowTile &r) {
        if (r.blocks == 0) {
            ra = rb = words_of(nullptr, 0);
            return;
        }
        // (first stage, as in moe_tiles, but per tile: a group's few rows of X
        // stay in L2.  16 experts of 4096 x 4096, 16 rows each: 109 -> 94 us)
        rot = BMN ? 0 : r.n0 / TNO % nk;
        const int64_t wbytes = (int64_t)p.N * p.K * 2;
        const uint8_t *wg = p.W + r.g * wbytes;
        const uint32_t have = p.rows ? (uint32_t)p.T : (uint32_t)min(r.mend - r.m0, 64);
        ra = words_of(p.rows ? p.X : p.X + (int64_t)r.m0 * lda, have * (uint32_t)lda);
        aoff = row < have ? row * (uint32_t)lda : kRowOOB;
        if constexpr (BMN) {
            rb = words_of(wg + r.n0 * 2, (uint32_t)(wbytes - r.n0 * 2));
        } else if constexpr (GATE) {
            // rows 32 wn + 16 u + q of the slot: row n0 + 16 wn + q of matrix u
            const int f = r.n0 + (lrow >> 5) * 16 + (lrow & 15);
            rb = words_of(wg, (uint32_t)wbytes);
            boff = f < p.ncols ? (uint32_t)((((lrow >> 4) & 1) * p.ncols + f) * lda) : kRowOOB;
        } else {
            rb = words_of(wg + (int64_t)r.n0 * lda, (uint32_t)(min(p.N - r.n0, 64) * lda));
            boff = (uint32_t)(lrow * lda);
        }
    };
    auto load = [&](int slot, int ks) {
        ks += rot;
        ks -= ks >= nk ? nk : 0;
        const uint32_t dst = slot * S::kSlot;
        const int kc = (int)kx + ks * kRowBytes;
        const bool in = kc < lda;
        dma<16>(ra, lds, dst + c.w * 1024, in ? aoff + kc : kRowOOB);
        if constexpr (BMN) {
#pragma unroll
            for (int q = 0; q < S::QB; ++q) {
                const uint32_t k = (uint32_t)(ks * 64 + 4 * q);            // four K-rows a wave-load
                dma<16>(rb, lds, dst + S::kA + (c.w * S::QB + q) * 1024,
                        k + 8 * c.w < (uint32_t)p.K ? boff + k * (uint32_t)ldb : kOOB);
            }
        } else {
            dma<16>(rb, lds, dst + S::kA + c.w * 1024, in ? boff + kc : kRowOOB);
        }
    };

    RowTile cur = find(tile), next{};
    fetch(cur);
    aim(cur);
#pragma unroll
    for (int f = 0; f < S::NS - 1; ++f) load(f, f);
    const int ar = 16 * wm + j;
    uint32_t fa = (uint32_t)(ar * kRowBytes + ((kgroup(g) ^ swz(ar)) << 4)), fb = S::kA + part_base<BMN>(c, wn);
    stage_barrier<S::kWait>();

    int rs = 0;               // slot the next stage reads
    for (;;) {
        tile += nwg;
        next = find(tile);
        fetch(next);
        f32x4 acc[NB] = {};
        for (int s = 0; s < nk; ++s) {
            int ks = s + S::NS - 1;
            if (ks >= nk) {
                ks -= nk;
                if (ks == 0) aim(next);
            }
            asm volatile("" : "+v"(kx), "+v"(fa), "+v"(fb));
            const uint32_t so = (uint32_t)(rs * S::kSlot);
            bf16x8 a[2], b[2][NB];
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
                a[kk] = lds_read<bf16x8>(lds, (fa ^ (uint32_t)(kk << 6)) + so);
#pragma unroll
                for (int u = 0; u < NB; ++u) b[kk][u] = part_frag<BMN>(lds, fb + so, kk, u >> 1, u & 1);
            }
            load(rs == 0 ? S::NS - 1 : rs - 1, ks);
#pragma unroll
            for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                for (int u = 0; u < NB; ++u)
                    acc[u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[kk][u], a[kk], acc[u], 0, 0, 0);
            stage_barrier<S::kWait>();
            rs = rs + 1 == S::NS ? 0 : rs + 1;
        }
        // lane: row 16 wm + l % 16, four columns of each block (block u: columns
        // 32 wn + 64 (u / 2) + 16 (u % 2) ..)
        const int r0 = cur.m0 + 16 * wm, left = __builtin_amdgcn_readfirstlane(max(0, min(16, cur.mend - r0)));
        const __amdgpu_buffer_rsrc_t rd = make_rsrc(p.D + (int64_t)r0 * p.ncols * 2, (uint32_t)left * (uint32_t)p.ncols * 2u);
#pragma unroll
        for (int u = 0; u < (GATE ? NB / 2 : NB); ++u) {
            float v[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] = GATE ? gated(acc[0][q], acc[1][q]) : acc[u][q];
            const int n = cur.n0 + (GATE ? 16 : 32) * wn + 64 * (u >> 1) + 16 * (u & 1) + 4 * g;
            const uint32_t at = (uint32_t)(j * p.ncols + n) * 2u;
            const uint32_t lo = pack_bf16(v[0], v[1]), hi = pack_bf16(v[2], v[3]);
            if (p.vec) {
                __builtin_amdgcn_raw_buffer_store_b64(u32x2{lo, hi}, rd, n < p.ncols ? at : kOOB, 0, kStoreCached);
            } else {
                const uint16_t w[4] = {(uint16_t)lo, (uint16_t)(lo >> 16), (uint16_t)hi, (uint16_t)(hi >> 16)};
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    __builtin_amdgcn_raw_buffer_store_b16(w[q], rd, n + q < p.ncols ? at + 2 * q : kOOB, 0, kStoreCached);
            }
        }
        if (next.blocks == 0) break;
        cur = next;
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // nothing is left to land in LDS
}

// ---------------------------------------------------------------------- dw

// The groups of E with work (all, or those with rows) into order, by their
// number of stages in steps of half an octave (two at least), the longest
// first: tiles are handed out in a snake, as the products' are, and end
// together the better the smaller the last ones are.  By one wave; returns how
// many.
__device__ __forceinline__ int sort_groups(uint16_t *order, const int32_t *first, int E, bool all, const Lane &c)
{
    auto step = [](int rows) { return (int)(__builtin_bit_cast(uint32_t, (float)max((rows + 63) / 64, 2)) >> 22); };
    int hi = step(0);
    const int lo = hi;
    for (int g = c.lane; g < E; g += 64) hi = max(hi, step(first[g + 1] - first[g]));
#pragma unroll
    for (int d = 32; d; d /= 2) hi = max(hi, __shfl_xor(hi, d));
    int n = 0;
    for (int k = hi; k >= lo; --k) {
        for (int g0 = 0; g0 < E; g0 += 64) {
            const int g = g0 + c.lane, rows = g < E ? first[g + 1] - first[g] : 0;
            const bool here = g < E && step(rows) == k && (all || rows > 0);
            const uint64_t who = __ballot(here);
            if (here) order[n + __popcll(who & (((uint64_t)1 << c.lane) - 1))] = (uint16_t)g;
            n += __popcll(who);
        }
    }
    return n;
}

// Tile columns along N handed out together: the 32 tiles that an XCD's
// workgroups hold together then read 8 + 4 parts of dY and X where all of 16
// and 2 took more (32 experts of 4096 x 2048, 1024 rows each: 556 -> 535 us).
constexpr int kDwBand = 8;

// GATHER: rows of X through p.rows.  F32: dW holds fp32.
//
// Gathered rows: a wave loads eight K-rows of X a stage.  Their indices reach
// LDS for eight stages at a time by one dword load of the wave's own (it
// waits for them by its own count, no barrier), into a buffer per parity of
// the tile for a tile's first eight stages and two in turn for later ones.
//
// 32768 rows of 32 uneven experts, 4096 x 2048: 542 us to bf16 (1.01 PFLOP/s)
// at 46 % of the matrix cores' cycles: 1.7 us a stage, and 5 us for each of a
// CU's 16 tiles, when all CUs write at once.  One expert of 16384 rows,
// 4096 x 4096: 413 us (1.33 PFLOP/s).
template <bool GATHER, bool F32>
__device__ __forceinline__ void dw_large(const MoeGemmDw &p, const Lane &c, uint8_t *lds, const int32_t *first,
                                         const uint16_t *order, int groups, uint32_t *rowbuf)
{
    constexpr int kStores = F32 ? 32 : 16;             // store instructions of a tile
    const int lda = p.N * 2, ldb = p.K * 2;            // bytes of a row of dY, of X
    const int tiles_n = (p.N + 255) / 256, tiles_k = (p.K + 255) / 256, per = tiles_n * tiles_k;
    const int ntiles = groups * per, nwg = gridDim.x, self = first_tile();
    if (self >= ntiles) return;

    struct Ref {
        int lo, hi, n0, k0, g, nk;
    };
    // past the last tile: no rows
    auto find = [&](int id) {
        Ref r{};
        r.nk = 2;
        if (id >= ntiles) return r;
        r.g = __builtin_amdgcn_readfirstlane((int)order[id / per]);
        r.lo = __builtin_amdgcn_readfirstlane(first[r.g]);
        r.hi = __builtin_amdgcn_readfirstlane(first[r.g + 1]);
        const int local = id % per;
        const int band = local / (kDwBand * tiles_k), wide = min(kDwBand, tiles_n - band * kDwBand);
        const int in = local - band * kDwBand * tiles_k;
        r.n0 = (band * kDwBand + in % wide) * 256;
        r.k0 = in / wide * 256;
        // the loads run up to two stages ahead: two at least
        r.nk = max(2, (r.hi - r.lo + 63) / 64);
        return r;
    };
    auto tile_of = [&](int round) { return snake(round, nwg, self); };
    Ref cur = find(self), next = cur;

    // What the loads read: stage lk of tile src, rows behind wa and wb.
    Ref src = cur;
    int lk = 0, left = 0, odd = 0;                     // rows of the stage; parity of src
    i32x4 wa, wb;
    uint32_t la = mn_part_lane(c, lda);
    uint32_t lb = mn_part_lane(c, GATHER ? 0 : ldb);
    uint32_t boff[2] = {};                             // gathered: the lane's offsets of its two wave-loads
    const i32x4 wr = words_of(p.rows, GATHER ? (uint32_t)p.M * 4u : 0u);
    auto batch = [&](const Ref &r, int b, int buffer) {
        if constexpr (GATHER) {
            const int m = r.lo + (8 * b + (c.lane >> 3)) * 64 + c.w * 8 + (c.lane & 7);
            dma<4>(wr, reinterpret_cast<uint8_t *>(rowbuf), c.w * 1024 + buffer * 256, (uint32_t)m * 4u);
        }
    };
    auto aim = [&] {
        const int m0 = src.lo + lk * 64;
        left = min(64, src.hi - m0);
        wa = words_of(p.dY + (int64_t)m0 * lda + src.n0 * 2, left > 0 ? (uint32_t)left * (uint32_t)lda - src.n0 * 2 : 0u);
        if constexpr (GATHER) {
            wb = words_of(p.X + src.k0 * 2, (uint32_t)p.T * (uint32_t)ldb - src.k0 * 2);
            const int b = lk >> 3;
            if ((lk & 7) == 0 && 8 * (b + 1) < src.nk) batch(src, b + 1, 2 + ((b + 1) & 1));
            const uint32_t *ix = rowbuf + c.w * 256 + (b == 0 ? odd : 2 + (b & 1)) * 64 + (lk & 7) * 8;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int i = q * 4 + (c.lane >> 4);
                const uint32_t row = ix[i];
                boff[q] = c.w * 8 + i < left && row < (uint32_t)p.T ? row * (uint32_t)ldb + lb : kRowOOB;
            }
        } else {
            wb = words_of(p.X + (int64_t)m0 * ldb + src.k0 * 2, left > 0 ? (uint32_t)left * (uint32_t)ldb - src.k0 * 2 : 0u);
        }
    };
    auto load = [&](int part, int slot) {
        const uint32_t dst = slot * kSlot + part * kPart + c.w * 2048;
        if (part == kALo || part == kAHi) {
            const uint32_t at = (uint32_t)(c.w * 8 * lda) + (part == kAHi ? 256 : 0);
            dma_group<true, 2>(wa, lds, dst, {la, la}, {at, at + (uint32_t)(4 * lda)});
            return;
        }
        if constexpr (GATHER) {
            dma_group<true, 4>(wb, lds, dst, {boff[0], boff[1], boff[0], boff[1]}, {0, 0, 256, 256}, kPart);
        } else {
            const uint32_t at = (uint32_t)(c.w * 8 * ldb), next = at + (uint32_t)(4 * ldb);
            dma_group<true, 4>(wb, lds, dst, {lb, lb, lb, lb}, {at, next, at + 256, next + 256}, kPart);
        }
    };

    batch(cur, 0, 0);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    aim();
    load(kALo, 0);
    load(kBLo, 0);
    load(kAHi, 0);
    lk = 1;
    aim();
    load(kALo, 1);
    load(kBLo, 1);
    uint32_t fa = part_base<true>(c, c.wm), fb = part_base<true>(c, c.wn);
    uint8_t *buf = lds + kStage + c.w * 2048;
    turn_end<kInFlight>();

    int slot = 0, stored = 0, parity = 0, round = 0;
    for (;;) {
        const int tile = tile_of(++round);
        next = find(tile);
        Acc acc;
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{};
        if (c.w >= 4) asm volatile("s_barrier" ::: "memory");      // one turn behind
#pragma clang loop unroll(disable)
        for (int s = 0; s < cur.nk; ++s) {
            asm volatile("" : "+v"(la), "+v"(lb), "+v"(fa), "+v"(fb));
            if (s == 0) batch(next, 0, parity ^ 1);
            core_stage<true, true, 2, 2>(
                acc, lds, fa, fb, slot, s == 0 ? stored : 0, load,
                [&] {
                    if (++lk == src.nk) {
                        // (from its third stage on a tile knows them landed)
                        if (GATHER && cur.nk < 3) asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
                        lk = 0;
                        src = next;
                        odd = parity ^ 1;
                    }
                    aim();
                },
                std::integral_constant<int, kStores>{});
            slot ^= 1;
        }
        if (c.w < 4) asm volatile("s_barrier" ::: "memory");
        DBS_FENCE();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r0 = cur.n0 + (2 * i + c.wm) * 32;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int k0 = cur.k0 + j * 128 + c.wn * 32;
                if constexpr (F32) {
                    // four consecutive columns a lane and 16 x 16 block
                    const int left = __builtin_amdgcn_readfirstlane(max(0, min(32, p.N - r0)));
                    const __amdgpu_buffer_rsrc_t rd = make_rsrc(p.dW + ((int64_t)cur.g * p.N + r0) * p.K * 4,
                                                                (uint32_t)left * (uint32_t)p.K * 4u);
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const int u = g >> 1, w = g & 1, k = k0 + 16 * w + 4 * (c.lane >> 4);
                        const uint32_t off =
                            k < p.K ? (uint32_t)((16 * u + (c.lane & 15)) * p.K + k) * 4u : kOOB;   // K % 8 == 0
                        f32x4 v = acc[2 * i + u][2 * j + w];
                        if (p.accumulate)
                            v += __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(rd, off, 0, 0));
                        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(i32x4, v), rd, off, 0, kStoreCached);
                    }
                } else {
                    store_block(buf, p.dW + (int64_t)cur.g * p.N * p.K * 2, p.K, r0, p.N, k0, p.K, 1, c,
                                [&](int u, int v, int q) { return acc[2 * i + u][2 * j + v][q]; });
                }
            }
        }
        stored = !p.accumulate;
        if (tile >= ntiles) break;
        cur = next;
        parity ^= 1;
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // nothing is left to land in LDS
}

// 64 (N) x 128 (K) tiles over a ring of five slots of 24 KiB, where there are so
// few 256 x 256 tiles that the longest sums decide: a stage costs 0.3 .. 0.55 us
// where the large tiles' costs 1.3 .. 2.3 for eight times the results.  8 waves
// (4 x 2) of 16 x 64.
//
// dY's part of a slot: 64 K-rows of 64 columns (128 bytes), wave-load w covers
// K-rows 8 w .. 8 w + 7; the transposed reads of two groups take 32 bytes of
// four K-rows each, groups 8 or 16 K-rows apart, and two K-rows share a bank
// line.  X's part as in the core.  Row indices as in dw_large, but a tile's
// first eight stages two tiles ahead: the loads run four stages ahead.
constexpr int kDwSlots = 5, kDwSlot = 64 * kRowBytes + 128 * kRowBytes;

template <bool GATHER, bool F32>
__device__ __forceinline__ void dw_small(const MoeGemmDw &p, const Lane &c, uint8_t *lds, const int32_t *first,
                                         const uint16_t *order, int groups)
{
    constexpr int NS = kDwSlots, kA = 64 * kRowBytes, kSlotD = kDwSlot, kWait = (NS - 2) * 3;
    uint32_t *rowbuf = reinterpret_cast<uint32_t *>(lds + NS * kSlotD);
    const int wm = c.w >> 1, wn = c.w & 1, j = c.lane & 15, g4 = c.lane >> 4;
    const int lda = p.N * 2, ldb = p.K * 2;            // bytes of a row of dY, of X
    const int tiles_n = (p.N + 63) / 64, tiles_k = (p.K + 127) / 128, per = tiles_n * tiles_k;
    const int ntiles = groups * per, nwg = gridDim.x, self = first_tile();
    if (self >= ntiles) return;

    struct Ref {
        int lo, hi, n0, k0, g, nk;
    };
    // past the last tile: no rows
    auto find = [&](int round) {
        Ref r{};
        r.nk = NS - 1;
        const int id = snake(round, nwg, self);
        if (id >= ntiles) return r;
        r.g = __builtin_amdgcn_readfirstlane((int)order[id / per]);
        r.lo = __builtin_amdgcn_readfirstlane(first[r.g]);
        r.hi = __builtin_amdgcn_readfirstlane(first[r.g + 1]);
        const int local = id % per;
        r.n0 = local % tiles_n * 64;
        r.k0 = local / tiles_n * 128;
        r.nk = max(NS - 1, (r.hi - r.lo + 63) / 64);
        return r;
    };

    // What the loads read: stage lk of tile src (its first indices in buffer fb0), rows behind wa and wb.
    Ref cur = find(0), next = find(1), src = cur;
    int lk = 0, fb0 = 0;
    i32x4 wa, wb;
    const int arow = 8 * c.w + (c.lane >> 3);
    const uint32_t la = (uint32_t)(arow * lda + (((c.lane & 7) ^ narrow_swz(arow)) << 4));
    const uint32_t lb = mn_part_lane(c, GATHER ? 0 : ldb) + (GATHER ? 0u : (uint32_t)(8 * c.w * ldb));
    const i32x4 wr = words_of(p.rows, GATHER ? (uint32_t)p.M * 4u : 0u);
    auto batch = [&](const Ref &r, int b, int buffer) {
        if constexpr (GATHER) {
            const int m = r.lo + (8 * b + (c.lane >> 3)) * 64 + c.w * 8 + (c.lane & 7);
            dma<4>(wr, reinterpret_cast<uint8_t *>(rowbuf), (c.w * 5 + buffer) * 256, (uint32_t)m * 4u);
        }
    };
    auto load = [&](int slot) {
        const int m0 = src.lo + lk * 64, left = min(64, src.hi - m0);
        const uint32_t dst = slot * kSlotD;
        uint32_t off[2];
        if constexpr (GATHER) {
            const int b = lk >> 3;
            if ((lk & 7) == 0 && 8 * (b + 1) < src.nk) batch(src, b + 1, 3 + ((b + 1) & 1));
            const uint32_t *ix = rowbuf + (c.w * 5 + (b == 0 ? fb0 : 3 + (b & 1))) * 64 + (lk & 7) * 8;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int i = q * 4 + g4;
                const uint32_t row = ix[i];
                off[q] = c.w * 8 + i < left && row < (uint32_t)p.T ? row * (uint32_t)ldb + lb : kRowOOB;
            }
            wb = words_of(p.X + src.k0 * 2, (uint32_t)p.T * (uint32_t)ldb - src.k0 * 2);
        } else {
            off[0] = lb;
            off[1] = lb + (uint32_t)(4 * ldb);
            wb = words_of(p.X + (int64_t)m0 * ldb + src.k0 * 2, left > 0 ? (uint32_t)left * (uint32_t)ldb - src.k0 * 2 : 0u);
        }
        wa = words_of(p.dY + (int64_t)m0 * lda + src.n0 * 2, left > 0 ? (uint32_t)left * (uint32_t)lda - src.n0 * 2 : 0u);
        dma<16>(wa, lds, dst + c.w * 1024, la);
#pragma unroll
        for (int q = 0; q < 2; ++q) dma<16>(wb, lds, dst + kA + (2 * c.w + q) * 1024, off[q]);
    };
    auto advance = [&](const Ref &then) {
        if (++lk == src.nk) {
            lk = 0;
            src = then;
            fb0 = fb0 == 2 ? 0 : fb0 + 1;
        }
    };

    batch(cur, 0, 0);
    batch(next, 0, 1);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    for (int f = 0; f < NS - 1; ++f) {
        load(f);
        advance(next);
    }
    uint32_t fa, fb = kA + part_base<true>(c, wn);
    {
        const int r = 8 * kgroup(g4) + (j >> 2);
        fa = (uint32_t)(r * kRowBytes + ((32 * wm + 8 * (j & 3)) ^ (narrow_swz(r) << 4)));
    }
    stage_barrier<kWait>();

    int rs = 0, round = 0;
    for (;;) {
        // the tile after the next one: its first indices go out a tile's stages ahead of their use
        const Ref after = find(round + 2);
        batch(after, 0, (round + 2) % 3);
        f32x4 acc[4] = {};
        for (int s = 0; s < cur.nk; ++s) {
            asm volatile("" : "+v"(fa), "+v"(fb));
            const uint32_t so = (uint32_t)(rs * kSlotD);
            bf16x8 a[2], b[2][4];
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
                typedef __attribute__((address_space(3))) i16x4 lds_i16x4;
                const uint8_t *x = lds + fa + so + kk * 32 * kRowBytes;
                const i32x2 lo = __builtin_bit_cast(i32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4 *)x));
                const i32x2 hi =
                    __builtin_bit_cast(i32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4 *)(x + 4 * kRowBytes)));
                a[kk] = __builtin_bit_cast(bf16x8, i32x4{lo[0], lo[1], hi[0], hi[1]});
#pragma unroll
                for (int u = 0; u < 4; ++u) b[kk][u] = part_frag<true>(lds, fb + so, kk, u >> 1, u & 1);
            }
            load(rs == 0 ? NS - 1 : rs - 1);
            // (past this tile's last stage the loads are the next one's, past that one's the one after's)
            advance(s + NS - 1 < cur.nk ? next : after);
#pragma unroll
            for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    acc[u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[kk][u], a[kk], acc[u], 0, 0, 0);
            stage_barrier<kWait>();
            rs = rs + 1 == NS ? 0 : rs + 1;
        }
        // lane: dW row 16 wm + l % 16, four columns of each block (block u: columns
        // 32 wn + 64 (u / 2) + 16 (u % 2) ..)
        constexpr int SZ = F32 ? 4 : 2;
        const int r0 = cur.n0 + 16 * wm, left = __builtin_amdgcn_readfirstlane(max(0, min(16, p.N - r0)));
        const __amdgpu_buffer_rsrc_t rd =
            make_rsrc(p.dW + ((int64_t)cur.g * p.N + r0) * p.K * SZ, (uint32_t)left * (uint32_t)p.K * (uint32_t)SZ);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int k = cur.k0 + 32 * wn + 64 * (u >> 1) + 16 * (u & 1) + 4 * g4;
            const uint32_t at = k < p.K ? (uint32_t)(j * p.K + k) * (uint32_t)SZ : kOOB;      // K % 8 == 0
            if constexpr (F32) {
                f32x4 v = acc[u];
                if (p.accumulate) v += __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(rd, at, 0, 0));
                __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(i32x4, v), rd, at, 0, kStoreCached);
            } else {
                __builtin_amdgcn_raw_buffer_store_b64(u32x2{pack_bf16(acc[u][0], acc[u][1]), pack_bf16(acc[u][2], acc[u][3])},
                                                      rd, at, 0, kStoreCached);
            }
        }
        if (snake(round + 1, nwg, self) >= ntiles) break;
        cur = next;
        next = after;
        ++round;
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // nothing is left to land in LDS
}

// Which of the two (moe_dw_small in moe.h): the stages and tiles of the busiest workgroup, in tenths
// of a microsecond as measured -- 1.6 us a stage of a large tile with all CUs
// at work, 1.3 along one long group, 5 to store it (9 in fp32) against 0.5,
// 0.35 and 1.  The groups decide: 19 experts of 848 x 632, 1024 rows each on
// average, even groups 43 us with large tiles and 56 with small ones, groups
// that differ by e^0.5 92 against 70; 8 of 1024 x 1024, 1024 rows, even 35 against 42,
// exponential 75 against 47; 32 of 4096 x 2048, 1024 rows 540 against 1180.  So
// it is made here, by every workgroup from the same offsets.
template <bool GATHER, bool F32>
__global__ __launch_bounds__(512, 1) void moe_dw(MoeGemmDw p)
{
    __shared__ __attribute__((aligned(1024))) uint8_t lds[kCoreLds];
    static_assert(kDwSlots * kDwSlot + 8 * 5 * 256 <= kCoreLds, "the small tiles' ring and row indices");
    __shared__ int32_t first[kMoeMaxExperts + 1];
    __shared__ uint16_t order[kMoeMaxExperts + 1];     // groups with tiles, the longest sums first
    __shared__ int32_t count, small;
    __shared__ uint32_t rowbuf[GATHER ? 8 * 256 : 1];
    const Lane c = lane_of();
    if (c.w == 0) {
        // (the table's second part, rows before a group, is not used)
        group_table<true>(first, order, p.offsets, p.E, p.M, c, [](int) { return 0; });
        wave_handover();
        const int n = sort_groups(order, first, p.E, !p.accumulate, c);
        wave_handover();
        int longest = 0, two = 0, four = 0;            // stages, at least two or four to a tile
        for (int i = c.lane; i < n; i += 64) {
            const int g = order[i], stages = (first[g + 1] - first[g] + 63) / 64;
            longest = max(longest, stages);
            two += max(stages, 2);
            four += max(stages, 4);
        }
#pragma unroll
        for (int d = 32; d; d /= 2) {
            longest = max(longest, __shfl_xor(longest, d));
            two += __shfl_xor(two, d);
            four += __shfl_xor(four, d);
        }
        if (c.lane == 0) {
            count = n;
            small = moe_dw_small(n, longest, two, four, p.N, p.K, F32, (int)gridDim.x);
        }
    }
    __syncthreads();
    const int groups = __builtin_amdgcn_readfirstlane(count);
    if (__builtin_amdgcn_readfirstlane(small)) dw_small<GATHER, F32>(p, c, lds, first, order, groups);
    else dw_large<GATHER, F32>(p, c, lds, first, order, groups, rowbuf);
}

// At most as many workgroups as there can be tiles of tm rows and tno columns.
dim3 tile_grid(const MoeGemm &p, int tm, int tno, int cus)
{
    const int64_t most = ((int64_t)p.M / tm + (p.M < p.E ? p.M : p.E)) * ((p.ncols + tno - 1) / tno);
    return dim3((uint32_t)(most < cus ? most : cus));
}

}  // namespace

hipError_t launch_moe_tiles(const MoeGemm &p, int rows, int cus, hipStream_t stream)
{
    const dim3 block(512);
    if (rows == 64) {
        const dim3 grid = tile_grid(p, 64, p.wmn ? Deep<true>::TN : p.gate ? Deep<false>::TN / 2 : Deep<false>::TN, cus);
        if (p.wmn) hipLaunchKernelGGL((moe_tiles_64<true, false>), grid, block, 0, stream, p);
        else if (p.gate) hipLaunchKernelGGL((moe_tiles_64<false, true>), grid, block, 0, stream, p);
        else hipLaunchKernelGGL((moe_tiles_64<false, false>), grid, block, 0, stream, p);
    } else {
        auto go = [&](auto tm) {
            constexpr int TM = decltype(tm)::value;
            const dim3 grid = tile_grid(p, TM, p.gate ? 128 : 256, cus);
            if (p.wmn) hipLaunchKernelGGL((moe_tiles<TM, true, false>), grid, block, 0, stream, p);
            else if (p.gate) hipLaunchKernelGGL((moe_tiles<TM, false, true>), grid, block, 0, stream, p);
            else hipLaunchKernelGGL((moe_tiles<TM, false, false>), grid, block, 0, stream, p);
        };
        if (rows == 256) go(std::integral_constant<int, 256>{});
        else go(std::integral_constant<int, 128>{});
    }
    return hipGetLastError();
}

hipError_t launch_moe_dw(const MoeGemmDw &p, int cus, hipStream_t stream)
{
    const dim3 grid((uint32_t)moe_dw_grid(p.E, p.N, p.K, cus)), block(512);
    auto go = [&](auto gather, auto f32) {
        hipLaunchKernelGGL((moe_dw<decltype(gather)::value, decltype(f32)::value>), grid, block, 0, stream, p);
        return hipGetLastError();
    };
    if (p.rows) return p.f32 ? go(std::true_type{}, std::true_type{}) : go(std::true_type{}, std::false_type{});
    return p.f32 ? go(std::false_type{}, std::true_type{}) : go(std::false_type{}, std::false_type{});
}

}  // namespace dbs
