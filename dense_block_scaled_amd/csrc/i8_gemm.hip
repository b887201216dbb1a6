// i8_gemm.hip -- gfx950 kernels of the products in 8-bit integers:
//
//   D[i, n] = sX[r] sW_g[n] sum_k X[r, k] W_g[n, k]      r = rows[i], i in group g (dense: one group, r = i)
//   D[i, f] = silu(h[f]) h[F + f]                        h = the first form's row, F = N / 2 (the gate)
//
// Codes are whole numbers in -128 .. 127, so the sums are exact in 32-bit integers up
// to K = 131071, in whatever order; a result is rounded where the sum becomes
// fp32 (above 2^24), at each scale and, once, to bf16.
//
// v_mfma_i32_16x16x64_i8 takes the bytes that the bf16 instruction of the experts'
// products takes (16 a lane, 64 of each of 16 rows) in the same cycles,
// so the core of moe_core.h serves unchanged with 128 K to a stage in place of 64; a
// lane's K are the same for both operands, whichever they are.
//
// * Scales.  256 row and 256 column scales of a tile are loaded to LDS when the
//   loads turn to it, two stages before the tile ahead of it ends, into one of two
//   places by the tile's parity: its results find them there without a wait.
// * Rows, bounds and the gate are the experts' products' (moe_gemm.hip).
//
// Tiles, from the fewest rows to the most (the rule is i8_tile in i8.cpp), and what bounds each:
//   16 x 16    W's rows straight into registers: 1 x 8192 x 8192 in 14.5 us, 4.6 TB/s of W from memory (11.9 and 5.6
//              where the caches have it)
//   16 x 64, 64 x 16 .. 64    a deep ring in LDS: 48 tokens to 8 of 128 experts of 2 768 x 4096, which meet 96 of
//              them, in 102 us, 5.9 TB/s of W; 48 x 8192 x 4096 in 11.0 (caches: 9.5), the way into the kernel and 16
//              stages' latency
//   128 x 64   128 x 11008 x 8192 in 32 us (caches: 26), 172 tiles
//   128 x 128  1024 x 4096 x 4096 in 22 us, a round of tiles: LDS (96 KiB read and 32 written a
//              stage, 1024 cycles at 128 bytes each, where the MFMAs take 512)
//   256 x 256  8192 x 8192 x 8192 in 400 .. 410 us, 2.7 Pop/s: power (MFMAs busy 68 % of the time at
//              1.9 GHz; codes of zero take 320 us)
#include "i8.h"
#include "moe_core.h"

namespace dbs {
namespace {

struct MulI8 {
    typedef i32x4 Sum;
    static __device__ __forceinline__ i32x4 mul(bf16x8 b, bf16x8 a, i32x4 c)
    {
        return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, b), __builtin_bit_cast(i32x4, a), c, 0, 0, 0);
    }
};

// Rows from .. to-1 of D are zero (those before the first group and behind the last).
__device__ __forceinline__ void zero_rows(const I8Gemm &p, int64_t from, int64_t to)
{
    const int64_t row = (int64_t)p.ldd * (p.f32 ? 4 : 2), bytes = (to - from) * row;
    uint8_t *z = p.D + from * row;
    const int64_t me = (int64_t)blockIdx.x * blockDim.x + threadIdx.x, all = (int64_t)gridDim.x * blockDim.x;
    if (p.vec)
        for (int64_t o = me * 16; o < bytes; o += all * 16) *reinterpret_cast<i32x4 *>(z + o) = i32x4{};
    else
        for (int64_t o = me * 2; o < bytes; o += all * 2) *reinterpret_cast<uint16_t *>(z + o) = 0;
}

// The tiles of a call: of groups by a table in LDS (moe_tiles.h), of the dense
// product's one group in the same order by arithmetic on its sizes, which saves
// small calls the way through LDS (three tiles of it before the first loads).
template <int TM>
struct Tiles {
    Table<TM> &tab;
    const I8Gemm &p;
    const Lane &c;
    int tiles_n, tno, count;

    __device__ __forceinline__ Tiles(Table<TM> &t, const I8Gemm &args, const Lane &lane, int width)
        : tab(t), p(args), c(lane), tiles_n((args.ncols + width - 1) / width), tno(width)
    {
        if (!p.offsets) {
            count = (p.M + TM - 1) / TM * tiles_n;
            return;
        }
        if constexpr (TM == 16) {
            if (c.w == 0) group_table<true>(tab.first, tab.whole, p.offsets, p.E, p.M, c, [](int rows) { return (rows + 15) / 16; });
            __syncthreads();
            zero_rows(p, 0, tab.first[0]);
            zero_rows(p, tab.first[p.E], p.M);
            count = same(tab.whole[p.E]) * tiles_n;
            return;
        }
        if (c.w == 0)
            group_table<true>(tab.first, tab.whole, p.offsets, p.E, p.M, c, [](int rows) { return Table<TM>::whole_of(rows); });
        else if (c.w < TM / 64)
            group_table<false>(tab.first, tab.rest[c.w - 1], p.offsets, p.E, p.M, c,
                               [&](int rows) { return Table<TM>::rest_of(rows, c.w); });
        __syncthreads();
        zero_rows(p, 0, tab.first[0]);
        zero_rows(p, tab.first[p.E], p.M);
        count = count_tiles(tab, p.E, tiles_n);
    }

    __device__ __forceinline__ RowTile operator()(int id) const
    {
        if constexpr (TM == 16) {
            RowTile r{};
            if (id >= count) return r;
            const int row_tile = id / tiles_n;
            r.blocks = 1;
            r.n0 = (id - row_tile * tiles_n) * tno;
            r.m0 = row_tile * 16;
            r.mend = p.M;
            if (p.offsets) {
                r.g = group_of(tab.whole, p.E, row_tile, c);
                r.m0 = same(tab.first[r.g]) + (row_tile - same(tab.whole[r.g])) * 16;
                r.mend = same(tab.first[r.g + 1]);
            }
            return r;
        }
        if (p.offsets)
            return find_tile(tab, p.E, count, tiles_n, tno, id, [&](const auto *at, int n) { return group_of(at, p.E, n, c); });
        RowTile r{};
        if (id >= count) return r;
        const int whole = Table<TM>::whole_of(p.M);
        r.mend = p.M;
        if (id < whole * tiles_n) {
            const int band = id / (kBand * tiles_n), rows = min(whole - band * kBand, kBand), in = id - band * kBand * tiles_n;
            r.m0 = (band * kBand + in % rows) * TM;
            r.n0 = in / rows * tno;
            r.blocks = TM / 64;
        } else {
            r.m0 = p.M / TM * TM;
            r.n0 = (id - whole * tiles_n) * tno;
            r.blocks = Table<TM>::blocks(p.M);
        }
        return r;
    }
};

// The workgroups that the tiles are spread over: no more than there are tiles,
// by eights, so that every XCD has its share of few (a grid is sized before the
// groups are known; 256 tiles by a grid of 512 kept to four XCDs: 11 us, not 7).
__device__ __forceinline__ int spread(int ntiles) { return min((int)gridDim.x, (ntiles + 7) & ~7); }

// As first_tile, over n workgroups; those behind them have no tile
__device__ __forceinline__ int first_of(int n, int ntiles)
{
    const int wg = blockIdx.x;
    return wg >= n ? ntiles : (n & 7) == 0 ? (wg & 7) * (n >> 3) + (wg >> 3) : wg;
}

// Four consecutive columns n .. n + 3 of a row as the type of D, at byte offset
// `at` (of column n) behind rd; columns past ncols are dropped.
template <bool F32>
__device__ __forceinline__ void store_four(__amdgpu_buffer_rsrc_t rd, const float (&v)[4], int n, int ncols, uint32_t at,
                                           int vec)
{
    if constexpr (F32) {
        if (vec) {
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(i32x4, f32x4{v[0], v[1], v[2], v[3]}), rd,
                                                   n < ncols ? at : kOOB, 0, kStoreCached);
        } else {
#pragma unroll
            for (int q = 0; q < 4; ++q)
                __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, v[q]), rd, n + q < ncols ? at + 4 * q : kOOB,
                                                      0, kStoreCached);
        }
    } else {
        const uint32_t lo = pack_bf16(v[0], v[1]), hi = pack_bf16(v[2], v[3]);
        if (vec) {
            __builtin_amdgcn_raw_buffer_store_b64(u32x2{lo, hi}, rd, n < ncols ? at : kOOB, 0, kStoreCached);
        } else {
            const uint16_t w[4] = {(uint16_t)lo, (uint16_t)(lo >> 16), (uint16_t)hi, (uint16_t)(hi >> 16)};
#pragma unroll
            for (int q = 0; q < 4; ++q)
                __builtin_amdgcn_raw_buffer_store_b16(w[q], rd, n + q < ncols ? at + 2 * q : kOOB, 0, kStoreCached);
        }
    }
}

// 16 rows r0 .. (up to mend) and 32 columns n0 .. of results, value(v, q): the
// lane's row l % 16, columns 16 v + 4 (l / 16) + q.  They go through the wave's
// 1 KiB buffer, 64 bytes of each row at a time (32 bf16, 16 fp32), so that a store
// takes whole pieces of 16 bytes, or neighbouring lanes write neighbouring columns
// (2047 x 4102 fp32 results, whose rows do not start on 16 bytes, element by
// element from the lanes that have them: 68 us where 2048 x 4096 take 48).
template <bool F32, class VALUE>
__device__ __forceinline__ void store_rows(uint8_t *buf, const I8Gemm &p, int r0, int mend, int n0, Lane c, VALUE &&value)
{
    constexpr int SZ = F32 ? 4 : 2, kCols = 64 / SZ;
    asm volatile("" : "+v"(c.lane));
    const int left = __builtin_amdgcn_readfirstlane(max(0, min(16, mend - r0)));
    const __amdgpu_buffer_rsrc_t rd = make_rsrc(p.D + (int64_t)r0 * p.ldd * SZ, (uint32_t)left * (uint32_t)p.ldd * (uint32_t)SZ);
    const int row = c.lane & 15, g = c.lane >> 4;
#pragma unroll
    for (int h = 0; h < (F32 ? 2 : 1); ++h) {
        const int nh = n0 + 16 * h;
        if (F32 && p.vec) {
            const float w[4] = {value(h, 0), value(h, 1), value(h, 2), value(h, 3)};
            store_four<true>(rd, w, nh + 4 * g, p.ncols, (uint32_t)(row * p.ldd + nh + 4 * g) * 4u, 1);
            continue;
        }
        wave_handover();                     // (the rows before have been read)
        if constexpr (F32) {
            *reinterpret_cast<f32x4 *>(buf + row * 64 + ((g ^ ((row >> 1) & 3)) << 4)) =
                f32x4{value(h, 0), value(h, 1), value(h, 2), value(h, 3)};
        } else {
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                const int col = 16 * v + 4 * g;
                *reinterpret_cast<u32x2 *>(buf + row * 64 + (((col >> 3) ^ ((row >> 1) & 3)) << 4) + 2 * (col & 4)) =
                    u32x2{pack_bf16(value(v, 0), value(v, 1)), pack_bf16(value(v, 2), value(v, 3))};
            }
        }
        wave_handover();
        if (!F32 && p.vec) {
            const int r = c.lane >> 2, ch = c.lane & 3, n = nh + ch * 8;
            const i32x4 v = *reinterpret_cast<const i32x4 *>(buf + r * 64 + 16 * (ch ^ ((r >> 1) & 3)));
            __builtin_amdgcn_raw_buffer_store_b128(v, rd, n < p.ncols ? (uint32_t)(r * p.ldd + n) * 2u : kOOB, 0, kStoreCached);
        } else {
            // lanes along the columns: 4 (fp32) or 2 (bf16) rows a store
            const int e = c.lane % kCols, n = nh + e;
#pragma unroll
            for (int q = 0; q < kCols / 4; ++q) {
                const int r = q * (64 / kCols) + c.lane / kCols, at = r * 64 + (((e * SZ >> 4) ^ ((r >> 1) & 3)) << 4) + (e * SZ & 15);
                const uint32_t to = n < p.ncols ? (uint32_t)(r * p.ldd + n) * (uint32_t)SZ : kOOB;
                if constexpr (F32)
                    __builtin_amdgcn_raw_buffer_store_b32(*reinterpret_cast<const uint32_t *>(buf + at), rd, to, 0, kStoreCached);
                else
                    __builtin_amdgcn_raw_buffer_store_b16(*reinterpret_cast<const uint16_t *>(buf + at), rd, to, 0, kStoreCached);
            }
        }
    }
}

// 256-row tiles by 256 rows of W; where a group has fewer rows left, the 64s of it that
// it has are multiplied.  GATE, F32: see the head of the file.
template <bool GATE, bool F32>
__global__ __launch_bounds__(512, 1) void i8_tiles(I8Gemm p)
{
    constexpr int TM = 256, kBufs = kStage, kLds = kStage + 8 * 1024;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[kLds];
    __shared__ Table<TM> tab;
    __shared__ uint32_t rowbuf[256];
    __shared__ __attribute__((aligned(16))) float scales[2][2][256];   // [parity of the tile][0: rows, 1: columns]
    constexpr int TNO = GATE ? 128 : 256;              // output columns of a tile
    constexpr int kStores = TM / 64 * (GATE ? 2 : F32 ? 8 : 4);        // store instructions of a whole tile (vec)

    Lane c = lane_of();
    const int lda = p.K;
    const Tiles<TM> tiles(tab, p, c, TNO);
    const int nwg = spread(tiles.count), self = first_of(nwg, tiles.count);
    if (self >= tiles.count) return;
    // at least three stages (the surplus reads zeros): the next tile's row
    // indices and scales land within a tile
    const int nk = max((p.K + kRowBytes - 1) / kRowBytes, 3);
    auto find = [&](int round) { return tiles(snake(round, nwg, self)); };

    // What the loads read: stage lk of the tile behind ra and rb.
    i32x4 ra, rb;
    uint32_t aoff[4];                     // the lane's row offsets in ra: A lo's two wave-loads, A hi's
    int f0 = 0, lk = 0, first_k = 0, parity = 0;
    uint32_t x4 = (uint32_t)(((c.lane & 7) ^ (c.lane >> 3)) << 4);
    uint32_t lb = (uint32_t)((c.lane >> 3) * lda);
    // Row indices of the tile `r` on their way into rowbuf (lanes past the
    // group's end load zeros, which aim does not use)
    auto fetch = [&](const RowTile &r) {
        if (c.w >= 4 || !p.rows) return;
        dma<4>(words_of(p.rows + r.m0, (uint32_t)max(min(r.mend - r.m0, TM), 0) * 4u), reinterpret_cast<uint8_t *>(rowbuf),
               c.w * 256, (uint32_t)(c.w * 256 + c.lane * 4));
    };
    auto aim = [&](const RowTile &r, int place) {
        // (the walk along K starts elsewhere per group and columns, as in moe_tiles)
        lk = first_k = (r.g * 7 + (r.n0 >> 11) * 5) % nk;
        if (r.blocks == 0) {
            ra = rb = words_of(nullptr, 0);
            return;
        }
        const int64_t wbytes = (int64_t)p.N * p.K;
        const uint8_t *wg = p.W + r.g * wbytes;
        f0 = r.n0;
        if constexpr (GATE)
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
        // 64 scales a wave: of rows (waves 0 .. 3), of columns (4 .. 7)
        const int m = (c.w & 3) * 64 + c.lane;
        const bool cols = c.w >= 4;
        const i32x4 rs = cols ? words_of(p.sW + (int64_t)r.g * p.N, (uint32_t)p.N * 4u)
                              : words_of(p.rows ? p.sX : p.sX + r.m0, have * 4u);
        uint32_t at;
        if (cols) at = (uint32_t)(GATE ? (m >> 7) * p.ncols + r.n0 + (m & 127) : r.n0 + m);
        else at = p.rows ? rowbuf[m] : (uint32_t)m;
        dma<4>(rs, reinterpret_cast<uint8_t *>(scales), place * 2048 + (cols ? 1024 : 0) + (c.w & 3) * 256,
               at < (uint32_t)(cols ? p.N : (int)have) ? at * 4u : kRowOOB);
    };
    auto load = [&](int part, int slot) {
        const uint32_t dst = slot * kSlot + part * kPart + c.w * 2048;
        // the lane's bytes of a row, and the least offset they lead to (past the row's end out of bounds)
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
            if constexpr (GATE) {
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
        if (lk == first_k) aim(next, parity ^ 1);
    };
    fetch(cur);
    if (p.rows) turn_end<0>();
    aim(cur, 0);
    load(kALo, 0);
    load(kBLo, 0);
    load(kAHi, 0);
    advance();
    load(kALo, 1);
    load(kBLo, 1);
    uint32_t fa = part_base<false>(c, c.wm), fb = part_base<false>(c, c.wn);
    uint8_t *buf = lds + kBufs + c.w * 1024;
    turn_end<kInFlight>();

    int slot = 0, round = 0, stored = 0;
    auto run = [&](auto nlo, auto nhi) {
        constexpr int NLO = decltype(nlo)::value, NHI = decltype(nhi)::value;
        Acc<MulI8> acc;
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = i32x4{};
        if (c.w >= 4) asm volatile("s_barrier" ::: "memory");      // one turn behind
#pragma clang loop unroll(disable)
        for (int s = 0; s < nk; ++s) {
            asm volatile("" : "+v"(x4), "+v"(lb), "+v"(fa), "+v"(fb));
            if (s == 0) fetch(next);
            core_stage<MulI8, false, false, NLO, NHI>(acc, lds, fa, fb, slot, s == 0 ? stored : 0, load, advance,
                                                      std::integral_constant<int, kStores>{});
            slot ^= 1;
        }
        if (c.w < 4) asm volatile("s_barrier" ::: "memory");
        DBS_FENCE();
        const float *sx = scales[parity][0], *sw = scales[parity][1];
        // the lane's columns' scales: [2 j + v]
        f32x4 sc[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int n = GATE ? 128 * (i >> 1) + 32 * c.wn : 64 * c.wn + 32 * (i >> 1);
            sc[i] = *reinterpret_cast<const f32x4 *>(sw + n + 16 * (i & 1) + 4 * (c.lane >> 4));
        }
#pragma unroll
        for (int i = 0; i < NLO + NHI; ++i) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int r = (2 * i + c.wm) * 32 + 16 * u;
                const float s = sx[r + (c.lane & 15)];
                auto scaled = [&](int j, int v, int q) { return (float)acc[2 * i + u][2 * j + v][q] * s * sc[2 * j + v][q]; };
                if constexpr (GATE) {
                    store_rows<F32>(buf, p, cur.m0 + r, cur.mend, cur.n0 + c.wn * 32, c,
                                    [&](int v, int q) { return gated(scaled(0, v, q), scaled(1, v, q)); });
                } else {
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        store_rows<F32>(buf, p, cur.m0 + r, cur.mend, cur.n0 + c.wn * 64 + j * 32, c,
                                        [&](int v, int q) { return scaled(j, v, q); });
                }
            }
        }
        stored = p.vec && NLO + NHI == TM / 64;
    };
    using I0 = std::integral_constant<int, 0>;
    using I1 = std::integral_constant<int, 1>;
    using I2 = std::integral_constant<int, 2>;
    for (;;) {
        next = find(++round);
        if (cur.blocks == 4) run(I2{}, I2{});
        else if (cur.blocks == 3) run(I2{}, I1{});
        else if (cur.blocks == 2) run(I2{}, I0{});
        else run(I1{}, I0{});
        if (next.blocks == 0) break;
        cur = next;
        parity ^= 1;
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // nothing is left to land in LDS
}

// Tiles over a deep ring (see moe_tiles_64).  64 rows by TN = 64, 32 or 16 rows of W for
// a few rows per group, where the time is the reading of W: what a CU can have
// under way is its LDS, over a latency of 1.2 us about 100 GB/s, so narrower
// tiles pay where wide ones leave CUs idle, although each reads all of X's rows.
// 16 rows by 64 where groups have no more: less of the ring goes to X, more to W (16 tokens
// to 8 of 64 experts of 2048 x 1408: 26.6 us, by 64 rows 29.0).
// 128 rows by 128, or by 64, where the large tiles are too few for the CUs.
//
// A stage is H times 128 bytes of every row.  8 waves: WM along the rows, the others
// along the columns or (KS = 2 or 4, where there are not enough of those to share
// out) each taking its part of a stage's k-steps, to be added at the end.  With the
// gate 16 gate rows of W and the 16 up rows that meet them alternate, and a wave
// has both.  Where the products count (PIPE) a wave reads a stage's blocks from LDS
// while it multiplies those of the stage before, whose slot is refilled at once
// (1024 x 4096 x 4096: one after the other 25.6 us, reads and loads in front
// of the products 25.2, between them 21.8 .. 23.7).  A tile's row
// indices are loaded two tiles ahead, its scales as in i8_tiles, all into LDS:
// the loads of the ring are waited for by count, and a load into registers would
// end that.
template <int TM_, int TN_, bool GATE>
struct Deep {
    static constexpr int TM = TM_, TN = TN_, H = TM == 128 ? 1 : TN == 16 ? 4 : 2;
    static constexpr int WM = TM == 16 ? 1 : TM == 128 && TN == 128 ? 2 : 4, RB = TM / 16 / WM;   // waves along the rows, blocks of 16 of each
    static constexpr int NB = (TM > 16 && TN >= 64) || GATE ? 2 : 1, WN = TN / 16 / NB, KS = 8 / WM / WN;
    static constexpr int kSteps = 2 * H / KS;                                  // k-steps of 64 bytes of a wave
    static constexpr int kA = TM * kRowBytes, kHalf = kA + TN * kRowBytes, kSlot = H * kHalf, kStageBytes = H * kRowBytes;
    static constexpr int NS = 131072 / kSlot;
    static constexpr bool PIPE = TM == 128;
    static constexpr int kAhead = PIPE ? NS : NS - 1;                          // stages that the loads are ahead
    static constexpr int kRows = TM < 64 ? 64 : TM;                            // of the tile's row indices and scales in LDS
    // wave-loads of a wave and 128 bytes of X's rows (TM = 16: the two of each go to four of the waves), of W's
    static constexpr int kLoadsA = TM / 64, kLoadsW = H * TN / 64, kLoads = H * kLoadsA + kLoadsW, kWait = (NS - 2) * kLoads;
    static constexpr int kRowsW = TN > 64 ? TN / 64 : 1;                       // wave-loads of W at rows of their own
    static constexpr int TNO = GATE ? TN / 2 : TN;
    static_assert(KS * WN * WM == 8 && 2 * H % KS == 0 && NS >= 3, "");
    static_assert(TM > 16 || H == 2, "four waves load X's rows");
};

// k-step kk (64 bytes) of the 16 rows 16 i further down than the lane's base: those
// change bits 1 and 2 of the swizzle
__device__ __forceinline__ bf16x8 deep_frag(const uint8_t *lds, uint32_t base, int kk, int i)
{
    return lds_read<bf16x8>(lds, (base ^ (uint32_t)((kk << 6) ^ ((i & 3) << 5))) + (uint32_t)(16 * i * kRowBytes));
}

template <int TM, int TN, bool GATE, bool F32>
__global__ __launch_bounds__(512, 1) void i8_tiles_deep(I8Gemm p)
{
    using S = Deep<TM, TN, GATE>;
    constexpr int RB = S::RB, NB = S::NB, KS = S::KS, H = S::H, TNO = S::TNO, SZ = F32 ? 4 : 2;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[S::NS * S::kSlot];
    __shared__ Table<TM> tab;
    __shared__ uint32_t rowbuf[2][S::kRows];
    // [parity of the tile]: rows' scales, then those of the tile's rows of W
    constexpr int kScales = S::kRows + (TN > 64 ? TN : 64);
    __shared__ __attribute__((aligned(16))) float scales[2][kScales];
    __shared__ __attribute__((aligned(16))) i32x4 part[TM == 128 ? 8 : KS > 1 ? (KS - 1) * S::WM * S::WN * NB : 1][64];

    const Lane c = lane_of();
    const int wm = c.w / (S::WN * KS), wn = c.w / KS % S::WN, ks = c.w % KS, j = c.lane & 15, g = c.lane >> 4;
    const int lda = p.K;
    const Tiles<TM> find(tab, p, c, TNO);
    const int nwg = spread(find.count);
    int tile = first_of(nwg, find.count);
    if (tile >= find.count) return;
    // more stages than the loads are ahead: they turn to the next tile behind a
    // barrier of this one, when the tile before's scales have been read.  (PIPE:
    // an even number, the two sets of registers take turns)
    int nk = max((p.K + S::kStageBytes - 1) / S::kStageBytes, S::kAhead + 1);
    if (S::PIPE) nk += nk & 1;

    // wave w loads rows 8 w .. (and 64 further down) of A; wave-load w + 8 q of W's: eight rows of one of the H parts
    i32x4 ra, rb;
    const int arow = 8 * (TM == 16 ? c.w & 1 : c.w) + (c.lane >> 3), wrow = 8 * (c.w % (TN / 8)) + (c.lane >> 3);
    int rot = 0;
    uint32_t aoff[S::kRows / 64], boff[S::kRowsW];
    uint32_t ax = (uint32_t)(((c.lane & 7) ^ swz(arow)) << 4), bx = (uint32_t)(((c.lane & 7) ^ swz(wrow)) << 4);   // the lane's chunks
    // (64 rows a wave; that the other waves have a load less under way waits for no fewer)
    auto fetch = [&](const RowTile &r, int place) {
        if (c.w >= S::kRows / 64 || !p.rows) return;
        dma<4>(words_of(p.rows + r.m0, (uint32_t)max(min(r.mend - r.m0, TM), 0) * 4u), reinterpret_cast<uint8_t *>(rowbuf),
               (place * S::kRows + c.w * 64) * 4, (uint32_t)(c.w * 64 + c.lane) * 4u);
    };
    auto row_of_w = [&](const RowTile &r, int e) { return ((e >> 4) & 1) * p.ncols + r.n0 + (e >> 5) * 16 + (e & 15); };
    // What the loads of W read
    auto aim_w = [&](const RowTile &r) {
        if (r.blocks == 0) {
            rb = words_of(nullptr, 0);
            return;
        }
        // The walk along K starts elsewhere per tile and group, or all read from few memory
        // channels; but not a step further for each tile, which keeps them together where rows
        // are 8 KiB apart (40 x 16384 x 8192 by 64 x 64: 39 us so, 30 all from the start, 27 like
        // this; 128 tokens to 2 of 16 experts of 4096 x 8192: 120, 96 like this)
        const int tn = r.n0 / TNO;
        rot = (7 * tn + 3 * (tn >> 3) + 5 * r.g) % nk;
        const int64_t wbytes = (int64_t)p.N * p.K;
        const uint8_t *wg = p.W + r.g * wbytes;
        rb = GATE ? words_of(wg, (uint32_t)wbytes) : words_of(wg + (int64_t)r.n0 * lda, (uint32_t)(min(p.N - r.n0, TN) * lda));
        // rows 32 i + 16 u + q of the slot, with the gate: row n0 + 16 i + q of matrix u
        auto there = [&](int e) { return r.n0 + (e >> 5) * 16 + (e & 15) < p.ncols; };
#pragma unroll
        for (int q = 0; q < S::kRowsW; ++q) {
            const int e = wrow + 64 * q;
            if constexpr (GATE) boff[q] = there(e) ? (uint32_t)(row_of_w(r, e) * lda) : kRowOOB;
            else boff[q] = (uint32_t)(e * lda);
        }
    };
    // Those of X, whose row indices are in rowbuf, and the scales
    auto aim_x = [&](const RowTile &r, int place) {
        if (r.blocks == 0) {
            ra = words_of(nullptr, 0);
            return;
        }
        const int left = min(r.mend - r.m0, TM);
        const uint32_t have = p.rows ? (uint32_t)p.T : (uint32_t)left;
        ra = words_of(p.rows ? p.X : p.X + (int64_t)r.m0 * lda, have * (uint32_t)lda);
#pragma unroll
        for (int q = 0; q < S::kRows / 64; ++q) {
            const int m = arow + 64 * q;
            const uint32_t row = p.rows ? rowbuf[place][m] : (uint32_t)m;
            aoff[q] = m < left && row < have ? row * (uint32_t)lda : kRowOOB;
        }
        if (c.w < S::kRows / 64) {
            const int m = c.w * 64 + c.lane;
            const uint32_t at = p.rows ? rowbuf[place][m] : (uint32_t)m;
            dma<4>(words_of(p.rows ? p.sX : p.sX + r.m0, have * 4u), reinterpret_cast<uint8_t *>(scales),
                   (place * kScales + c.w * 64) * 4, at < have ? at * 4u : kRowOOB);
        } else if (c.w < S::kRows / 64 + (TN + 63) / 64) {
            const int e = (c.w - S::kRows / 64) * 64 + c.lane, at = GATE ? row_of_w(r, e) : r.n0 + e;
            dma<4>(words_of(p.sW + (int64_t)r.g * p.N, (uint32_t)p.N * 4u), reinterpret_cast<uint8_t *>(scales),
                   (place * kScales + c.w * 64) * 4, e < TN && at < p.N ? (uint32_t)at * 4u : kRowOOB);
        }
    };
    // Wave-load q of the wave's kLoads of a stage at `k0` of the row: X's, then W's
    auto load_one = [&](int q, int slot, int k0) {
        const uint32_t dst = slot * S::kSlot;
        if (q < H * S::kLoadsA) {
            constexpr int kEach = S::kLoadsA > 0 ? S::kLoadsA : 1;
            const int h = q / kEach, r = q % kEach, kc = (int)ax + k0 + h * kRowBytes;
            dma<16>(ra, lds, dst + h * S::kHalf + (c.w + 8 * r) * 1024, kc < lda ? aoff[r] + kc : kRowOOB);
        } else {
            q -= H * S::kLoadsA;
            const int i = c.w + 8 * q, h = i / (TN / 8), kc = (int)bx + k0 + h * kRowBytes;
            dma<16>(rb, lds, dst + h * S::kHalf + S::kA + i % (TN / 8) * 1024,
                    kc < lda ? boff[S::kRowsW > 1 ? q : 0] + kc : kRowOOB);
        }
    };
    auto start_of = [&](int ks) {
        ks += rot;
        return (ks >= nk ? ks - nk : ks) * S::kStageBytes;
    };
    constexpr int kOfX = H * S::kLoadsA;
    auto load_w = [&](int slot, int ks) {
#pragma unroll
        for (int q = kOfX; q < S::kLoads; ++q) load_one(q, slot, start_of(ks));
    };
    auto load_x = [&](int slot, int ks) {
        const int k0 = start_of(ks);
#pragma unroll
        for (int q = 0; q < kOfX; ++q) load_one(q, slot, k0);
        if constexpr (TM == 16) {
            if (c.w < 4) {
                const int kc = (int)ax + k0 + (c.w >> 1) * kRowBytes;
                dma<16>(ra, lds, slot * S::kSlot + (c.w >> 1) * S::kHalf + (c.w & 1) * 1024, kc < lda ? aoff[0] + kc : kRowOOB);
            }
        }
    };
    // Until all but the loads of the last `stages` stages have landed (every wave waits for
    // its own: four of TM = 16's have one more in each stage)
    auto barrier = [&](auto stages) {
        constexpr int n = decltype(stages)::value;
        if (TM == 16 && c.w < 4) stage_barrier<n * (S::kLoads + (TM == 16))>();
        else stage_barrier<n * S::kLoads>();
    };
    using Ring = std::integral_constant<int, S::NS - 2>;

    int parity = 0;
    RowTile cur = find(tile);
    fetch(cur, 0);
    RowTile next = find(tile + nwg);
    fetch(next, 1);
    // (W's loads of two stages do not wait for the row indices)
    aim_w(cur);
    load_w(0, 0);
    load_w(1, 1);
    if (p.rows) turn_end<2 * S::kLoadsW>();
    aim_x(cur, 0);
    load_x(0, 0);
    load_x(1, 1);
#pragma unroll
    for (int f = 2; f < S::kAhead; ++f) {
        load_w(f, f);
        load_x(f, f);
    }
    const int ar = 16 * RB * wm + j, br = 16 * NB * wn + j;
    uint32_t fa = (uint32_t)(ar * kRowBytes + ((kgroup(g) ^ swz(ar)) << 4));
    uint32_t fb = (uint32_t)(S::kA + br * kRowBytes + ((kgroup(g) ^ swz(br)) << 4));
    struct Blocks {
        bf16x8 a[S::kSteps][RB], b[S::kSteps][NB];
    };
    // read n of the kReads of a stage
    constexpr int kReads = S::kSteps * (RB + NB);
    auto read_one = [&](Blocks &f, int slot, int n) {
        const int kk = n / (RB + NB), i = n % (RB + NB);
        const int step = ks * S::kSteps + kk;
        const uint32_t from = (uint32_t)(slot * S::kSlot + (step >> 1) * S::kHalf);
        if (i < NB) f.b[kk][i] = deep_frag(lds, fb + from, step & 1, i);
        else f.a[kk][i - NB] = deep_frag(lds, fa + from, step & 1, i - NB);
    };
    auto read = [&](Blocks &f, int slot) {
#pragma unroll
        for (int n = 0; n < kReads; ++n) read_one(f, slot, n);
    };
    Blocks even, odd;
    if constexpr (S::PIPE) {
        stage_barrier<S::kWait>();
        read(even, 0);
        stage_barrier<S::kWait>();
    } else {
        barrier(std::integral_constant<int, S::NS - 3>{});   // (stage 1's W came before stage 0's X)
    }

    int rs = 0;               // slot of the stage
    for (;;) {
        tile += nwg;
        // (this tile's row indices have been read: their place is the tile's after the next one)
        const RowTile after = find(tile + nwg);
        fetch(after, parity);
        const bool busy = cur.m0 + 16 * RB * wm < cur.mend;        // the wave has rows
        i32x4 acc[RB][NB];
#pragma unroll
        for (int i = 0; i < RB; ++i)
#pragma unroll
            for (int u = 0; u < NB; ++u) acc[i][u] = i32x4{};
        auto multiply = [&](const Blocks &f) {
#pragma unroll
            for (int kk = 0; kk < S::kSteps; ++kk)
#pragma unroll
                for (int i = 0; i < RB; ++i)
#pragma unroll
                    for (int u = 0; u < NB; ++u) acc[i][u] = MulI8::mul(f.b[kk][u], f.a[kk][i], acc[i][u]);
        };
        auto ahead = [&](int s) {
            int ks = s + S::kAhead;
            if (ks >= nk) {
                ks -= nk;
                if (ks == 0) {
                    aim_w(next);
                    aim_x(next, parity ^ 1);
                }
            }
            asm volatile("" : "+v"(ax), "+v"(bx), "+v"(fa), "+v"(fb));
            return ks;
        };
        if constexpr (S::PIPE) {
            auto stage = [&](const Blocks &now, Blocks &then, int s) {
                const int ks = ahead(s), after_rs = rs + 1 == S::NS ? 0 : rs + 1;
                const int k0 = start_of(ks);
                // reads and loads stand between the products, which they would hold back in front of them
                constexpr int kAll = S::kSteps * RB * NB;
#pragma unroll
                for (int m = 0; m < kAll; ++m) {
                    const int kk = m / (RB * NB), i = m / NB % RB, u = m % NB;
                    acc[i][u] = MulI8::mul(now.b[kk][u], now.a[kk][i], acc[i][u]);
                    DBS_FENCE();
#pragma unroll
                    for (int n = 0; n < kReads; ++n)
                        if (m == n * kAll / (kReads > kAll ? kReads : kAll)) read_one(then, after_rs, n);
#pragma unroll
                    for (int q = 0; q < S::kLoads; ++q)
                        if (m == ((q + 1) * kAll - 1) / S::kLoads) load_one(q, rs, k0);
                    DBS_FENCE();
                }
                stage_barrier<S::kWait>();
                rs = after_rs;
            };
            for (int s = 0; s < nk; s += 2) {
                stage(even, odd, s);
                stage(odd, even, s + 1);
            }
        } else {
            for (int s = 0; s < nk; ++s) {
                const int ks = ahead(s);
                read(even, rs);
                load_w(rs == 0 ? S::NS - 1 : rs - 1, ks);
                load_x(rs == 0 ? S::NS - 1 : rs - 1, ks);
                multiply(even);
                barrier(Ring{});
                rs = rs + 1 == S::NS ? 0 : rs + 1;
            }
        }
        if constexpr (KS > 1) {
            // (read before the next tile's stages end, written behind them)
            const int at = (S::WN * wm + wn) * NB;
            constexpr int kBlocks = S::WM * S::WN * NB;
            if (ks) {
#pragma unroll
                for (int u = 0; u < NB; ++u) part[(ks - 1) * kBlocks + at + u][c.lane] = acc[0][u];
            }
            asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
            if (!ks) {
#pragma unroll
                for (int h = 0; h < KS - 1; ++h)
#pragma unroll
                    for (int u = 0; u < NB; ++u) acc[0][u] += part[h * kBlocks + at + u][c.lane];
            }
        }
        if (!ks && busy) {
            // lane: rows l % 16 of each block, four columns of each
            f32x4 sw[NB];
#pragma unroll
            for (int u = 0; u < NB; ++u)
                sw[u] = *reinterpret_cast<const f32x4 *>(&scales[parity][S::kRows + 16 * NB * wn + 16 * u + 4 * g]);
#pragma unroll
            for (int i = 0; i < RB; ++i) {
                const int r0 = cur.m0 + 16 * (RB * wm + i);
                const float sx = scales[parity][ar + 16 * i];
                auto scaled = [&](int u, int q) { return (float)acc[i][u][q] * sx * sw[u][q]; };
                if constexpr (TM == 128 && !GATE) {
                    store_rows<F32>(reinterpret_cast<uint8_t *>(part[c.w]), p, r0, cur.mend, cur.n0 + 32 * wn, c, scaled);
                } else {
                    const int left = __builtin_amdgcn_readfirstlane(max(0, min(16, cur.mend - r0)));
                    const __amdgpu_buffer_rsrc_t rd =
                        make_rsrc(p.D + (int64_t)r0 * p.ldd * SZ, (uint32_t)left * (uint32_t)p.ldd * (uint32_t)SZ);
#pragma unroll
                    for (int u = 0; u < (GATE ? 1 : NB); ++u) {
                        float v[4];
#pragma unroll
                        for (int q = 0; q < 4; ++q) v[q] = GATE ? gated(scaled(0, q), scaled(NB - 1, q)) : scaled(u, q);
                        const int n = cur.n0 + (GATE ? 16 : 16 * NB) * wn + 16 * u + 4 * g;
                        store_four<F32>(rd, v, n, p.ncols, (uint32_t)(j * p.ldd + n) * (uint32_t)SZ, p.vec);
                    }
                }
            }
        }
        if (next.blocks == 0) break;
        cur = next;
        next = after;
        parity ^= 1;
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // nothing is left to land in LDS
}

// Few rows: 16 rows and 16 columns a workgroup (with the gate 16 gate columns and
// the 16 up columns that meet them), whose 8 waves share out K: every wave sums
// its part, from fragments loaded straight into registers (no wave reads what
// another does, so LDS would only be a detour), and the parts meet in LDS at the
// end, exact in whatever order.  So a matrix of a few thousand rows occupies
// every CU, and a walk along K is an eighth as long.  Two workgroups a CU fill
// each other's pauses, and the loads of the next tile go out before this one's
// parts meet.
constexpr int kRowsUnroll = 4;                   // k-steps of 64 bytes loaded together, twice

template <bool GATE, bool F32>
__global__ __launch_bounds__(512, 4) void i8_rows(I8Gemm p)
{
    constexpr int U = GATE ? 3 : kRowsUnroll, C = GATE ? 2 : 1, SZ = F32 ? 4 : 2;
    __shared__ __attribute__((aligned(16))) i32x4 part[C][8][64];
    __shared__ int32_t first[kMoeMaxExperts + 1], at[kMoeMaxExperts + 1];
    const Lane c = lane_of();
    const int j = c.lane & 15, g = c.lane >> 4;
    const int tiles_n = (p.ncols + 15) / 16;
    auto tiles_of = [](int rows) { return (rows + 15) / 16; };
    int row_tiles = tiles_of(p.M);               // (of the dense product)
    if (p.offsets) {
        if (c.w == 0) group_table<true>(first, at, p.offsets, p.E, p.M, c, tiles_of);
        __syncthreads();
        zero_rows(p, 0, first[0]);
        zero_rows(p, first[p.E], p.M);
        row_tiles = same(at[p.E]);
    }
    const int ntiles = row_tiles * tiles_n, nwg = spread(ntiles);
    int tile = first_of(nwg, ntiles);
    if (tile >= ntiles) return;
    // the wave's k-steps; the lane's end of them
    const int steps = (p.K + 63) / 64, each = (steps + 7) / 8, s0 = c.w * each, s1 = min(s0 + each, steps);
    const int kend = min(s1 * 64, p.K - 16 * g);

    struct Ref {
        int m0, left, n0, grp;
        uint32_t row;                            // the lane's row of X
    };
    auto find = [&](int id) {
        Ref t{};
        if (id >= ntiles) return t;
        const int row_tile = id / tiles_n;
        t.n0 = (id - row_tile * tiles_n) * 16;
        t.m0 = row_tile * 16;
        int end = p.M;
        if (p.offsets) {
            t.grp = group_of(at, p.E, row_tile, c);
            t.m0 = same(first[t.grp]) + (row_tile - same(at[t.grp])) * 16;
            end = same(first[t.grp + 1]);
        }
        t.left = min(end - t.m0, 16);
        t.row = j < t.left ? (p.rows ? (uint32_t)p.rows[t.m0 + j] : (uint32_t)j) : ~0u;
        return t;
    };
    // What the loads read: the tile behind ra and rb.
    __amdgpu_buffer_rsrc_t ra, rb;
    uint32_t aoff, boff[C];
    auto aim = [&](const Ref &t) {
        const int64_t wbytes = (int64_t)p.N * p.K;
        const uint8_t *wg = p.W + t.grp * wbytes;
        const uint32_t have = p.rows ? (uint32_t)p.T : (uint32_t)t.left;
        ra = make_rsrc(p.rows ? p.X : p.X + (int64_t)t.m0 * p.K, have * (uint32_t)p.K);
        rb = GATE ? make_rsrc(wg, (uint32_t)wbytes)
                  : make_rsrc(wg + (int64_t)t.n0 * p.K, (uint32_t)max(min(p.N - t.n0, 16), 0) * (uint32_t)p.K);
        aoff = t.row < have ? t.row * (uint32_t)p.K + 16 * g : kRowOOB;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            if constexpr (GATE) boff[i] = t.n0 + j < p.ncols ? (uint32_t)(i * p.ncols + t.n0 + j) * (uint32_t)p.K + 16 * g : kRowOOB;
            else boff[i] = (uint32_t)j * (uint32_t)p.K + 16 * g;
        }
    };
    bf16x8 a[2][U], b[2][U][C];
    auto load = [&](int place, int s) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = (s + u) * 64;
            const bool in = k < kend;            // (past the wave's part or the row's end: out of bounds, zero)
#pragma unroll
            for (int i = 0; i < C; ++i)
                b[place][u][i] =
                    __builtin_bit_cast(bf16x8, __builtin_amdgcn_raw_buffer_load_b128(rb, in ? boff[i] + k : kRowOOB, 0, 0));
            a[place][u] = __builtin_bit_cast(bf16x8, __builtin_amdgcn_raw_buffer_load_b128(ra, in ? aoff + k : kRowOOB, 0, 0));
        }
        DBS_FENCE();                             // (all of them before the products of those before)
    };
    i32x4 acc[C];
    auto mul = [&](int place) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < C; ++i) acc[i] = MulI8::mul(b[place][u][i], a[place][u], acc[i]);
        DBS_FENCE();
    };

    Ref cur = find(tile);
    aim(cur);
    load(0, s0);
    for (;;) {
        tile += nwg;
        const bool more = tile < ntiles;
        const Ref next = find(tile);
        // the scales that the results of this tile meet (by the first wave)
        const int n = cur.n0 + 4 * g;
        const uint32_t have = p.rows ? (uint32_t)p.T : (uint32_t)cur.left;
        float sx = 0.0f, sw[C][4] = {};
        if (c.w == 0) {
            const __amdgpu_buffer_rsrc_t rx = make_rsrc(p.rows ? p.sX : p.sX + cur.m0, have * 4u);
            const __amdgpu_buffer_rsrc_t rw = make_rsrc(p.sW + (int64_t)cur.grp * p.N, (uint32_t)p.N * 4u);
            sx = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rx, cur.row < have ? cur.row * 4u : kRowOOB, 0, 0));
#pragma unroll
            for (int h = 0; h < C; ++h)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    sw[h][q] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(
                                                             rw, n + q < p.ncols ? (uint32_t)(h * p.ncols + n + q) * 4u : kRowOOB, 0, 0));
        }
#pragma unroll
        for (int i = 0; i < C; ++i) acc[i] = i32x4{};
        int s = s0;
        for (; s + 2 * U < s1; s += 2 * U) {
            load(1, s + U);
            mul(0);
            load(0, s + 2 * U);
            mul(1);
        }
        load(1, s + U);
        mul(0);
        if (more) {
            aim(next);
            load(0, s0);
        }
        mul(1);
#pragma unroll
        for (int i = 0; i < C; ++i) part[i][c.w][c.lane] = acc[i];
        __syncthreads();
        if (c.w == 0) {
            float h[C][4];
#pragma unroll
            for (int i = 0; i < C; ++i) {
                i32x4 sum = {};
#pragma unroll
                for (int w = 0; w < 8; ++w) sum += part[i][w][c.lane];
#pragma unroll
                for (int q = 0; q < 4; ++q) h[i][q] = (float)sum[q] * sx * sw[i][q];
            }
            float v[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] = GATE ? gated(h[0][q], h[C - 1][q]) : h[0][q];
            const __amdgpu_buffer_rsrc_t rd =
                make_rsrc(p.D + (int64_t)cur.m0 * p.ldd * SZ, (uint32_t)cur.left * (uint32_t)p.ldd * (uint32_t)SZ);
            store_four<F32>(rd, v, n, p.ncols, (uint32_t)(j * p.ldd + n) * (uint32_t)SZ, p.vec);
        }
        if (!more) break;
        __syncthreads();                         // (the parts have been read)
        cur = next;
    }
}

// At most as many workgroups as there can be tiles of tm rows and tno columns.
dim3 tile_grid(const I8Gemm &p, int tm, int tno, int cus)
{
    const int64_t most = ((int64_t)p.M / tm + (p.M < p.E ? p.M : p.E)) * ((p.ncols + tno - 1) / tno);
    return dim3((uint32_t)(most < cus ? most : cus));
}

}  // namespace

hipError_t launch_i8_tiles(const I8Gemm &p, I8Tile t, int cus, hipStream_t stream)
{
    const dim3 block(512);
    if (t.cols == 16 && t.rows == 16) {
        const dim3 grid = tile_grid(p, 16, 16, 2 * cus);
        if (p.gate) hipLaunchKernelGGL((i8_rows<true, false>), grid, block, 0, stream, p);
        else if (p.f32) hipLaunchKernelGGL((i8_rows<false, true>), grid, block, 0, stream, p);
        else hipLaunchKernelGGL((i8_rows<false, false>), grid, block, 0, stream, p);
    } else if (t.cols <= 128) {
        auto go = [&](auto tm, auto tn) {
            constexpr int TM = decltype(tm)::value, TN = decltype(tn)::value;
            const dim3 grid = tile_grid(p, TM, p.gate ? TN / 2 : TN, cus);
            if constexpr (TN >= 32 && (TM < 128 || TN == 128)) {      // (the others are of the dense product)
                if (p.gate) {
                    hipLaunchKernelGGL((i8_tiles_deep<TM, TN, true, false>), grid, block, 0, stream, p);
                    return;
                }
            }
            if (p.f32) hipLaunchKernelGGL((i8_tiles_deep<TM, TN, false, true>), grid, block, 0, stream, p);
            else hipLaunchKernelGGL((i8_tiles_deep<TM, TN, false, false>), grid, block, 0, stream, p);
        };
        using I64 = std::integral_constant<int, 64>;
        using I128 = std::integral_constant<int, 128>;
        if (t.rows == 128 && t.cols == 128) go(I128{}, I128{});
        else if (t.rows == 128) go(I128{}, I64{});
        else if (t.rows == 16) go(std::integral_constant<int, 16>{}, I64{});
        else if (t.cols == 64) go(I64{}, I64{});
        else if (t.cols == 32 || p.gate) go(I64{}, std::integral_constant<int, 32>{});
        else go(I64{}, std::integral_constant<int, 16>{});
    } else {
        const dim3 grid = tile_grid(p, 256, p.gate ? 128 : 256, cus);
        if (p.gate) hipLaunchKernelGGL((i8_tiles<true, false>), grid, block, 0, stream, p);
        else if (p.f32) hipLaunchKernelGGL((i8_tiles<false, true>), grid, block, 0, stream, p);
        else hipLaunchKernelGGL((i8_tiles<false, false>), grid, block, 0, stream, p);
    }
    return hipGetLastError();
}

}  // namespace dbs
