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

template <int TM>
__device__ __forceinline__ void fill_table(Table<TM> &tab, const I8Gemm &p, const Lane &c)
{
    if (!p.offsets) {
        if (threadIdx.x == 0) {
            tab.first[0] = tab.whole[0] = 0;
            tab.first[1] = p.M;
            tab.whole[1] = Table<TM>::whole_of(p.M);
#pragma unroll
            for (int b = 0; b < Table<TM>::kRests; ++b) {
                tab.rest[b][0] = 0;
                tab.rest[b][1] = (uint16_t)Table<TM>::rest_of(p.M, b + 1);
            }
        }
    } else if (c.w == 0) {
        group_table<true>(tab.first, tab.whole, p.offsets, p.E, p.M, c, [](int rows) { return Table<TM>::whole_of(rows); });
    } else if (c.w < TM / 64) {
        group_table<false>(tab.first, tab.rest[c.w - 1], p.offsets, p.E, p.M, c,
                           [&](int rows) { return Table<TM>::rest_of(rows, c.w); });
    }
}

// Rows from .. to-1 of D are zero (those before the first group and behind the last).
__device__ __forceinline__ void zero_rows(const I8Gemm &p, int64_t from, int64_t to)
{
    const int64_t row = (int64_t)p.ncols * (p.f32 ? 4 : 2), bytes = (to - from) * row;
    uint8_t *z = p.D + from * row;
    const int64_t me = (int64_t)blockIdx.x * blockDim.x + threadIdx.x, all = (int64_t)gridDim.x * blockDim.x;
    if (p.vec)
        for (int64_t o = me * 16; o < bytes; o += all * 16) *reinterpret_cast<i32x4 *>(z + o) = i32x4{};
    else
        for (int64_t o = me * 2; o < bytes; o += all * 2) *reinterpret_cast<uint16_t *>(z + o) = 0;
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
// lane's row l % 16, columns 16 v + 4 (l / 16) + q.  bf16 rows that take
// 16-byte stores go through the wave's 1 KiB buffer (see store_block).
template <bool F32, class VALUE>
__device__ __forceinline__ void store_rows(uint8_t *buf, const I8Gemm &p, int r0, int mend, int n0, Lane c, VALUE &&value)
{
    constexpr int SZ = F32 ? 4 : 2;
    asm volatile("" : "+v"(c.lane));
    const int left = __builtin_amdgcn_readfirstlane(max(0, min(16, mend - r0)));
    const __amdgpu_buffer_rsrc_t rd = make_rsrc(p.D + (int64_t)r0 * p.ncols * SZ, (uint32_t)left * (uint32_t)p.ncols * (uint32_t)SZ);
    const int row = c.lane & 15, col0 = 4 * (c.lane >> 4);
    if (!F32 && p.vec) {
        wave_handover();                     // (the rows before have been read)
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            const int col = 16 * v + col0;
            *reinterpret_cast<u32x2 *>(buf + row * 64 + (((col >> 3) ^ ((row >> 1) & 3)) << 4) + 2 * (col & 4)) =
                u32x2{pack_bf16(value(v, 0), value(v, 1)), pack_bf16(value(v, 2), value(v, 3))};
        }
        wave_handover();
        const int r = c.lane >> 2, ch = c.lane & 3, n = n0 + ch * 8;
        const i32x4 v = *reinterpret_cast<const i32x4 *>(buf + r * 64 + 16 * (ch ^ ((r >> 1) & 3)));
        __builtin_amdgcn_raw_buffer_store_b128(v, rd, n < p.ncols ? (uint32_t)(r * p.ncols + n) * 2u : kOOB, 0, kStoreCached);
    } else {
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            const int n = n0 + 16 * v + col0;
            const float w[4] = {value(v, 0), value(v, 1), value(v, 2), value(v, 3)};
            store_four<F32>(rd, w, n, p.ncols, (uint32_t)(row * p.ncols + n) * (uint32_t)SZ, p.vec);
        }
    }
}

// 256-row tiles, or of 128 rows (TM) where a call has too few of the large ones
// for the CUs: the same stages, A's upper half filled with zeros and not
// multiplied.  GATE, F32: see the head of the file.
template <int TM, bool GATE, bool F32>
__global__ __launch_bounds__(512, 1) void i8_tiles(I8Gemm p)
{
    constexpr int kBufs = kStage, kLds = kStage + 8 * 1024;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[kLds];
    __shared__ Table<TM> tab;
    __shared__ uint32_t rowbuf[256];
    __shared__ __attribute__((aligned(16))) float scales[2][2][256];   // [parity of the tile][0: rows, 1: columns]
    constexpr int TNO = GATE ? 128 : 256;              // output columns of a tile
    constexpr int kStores = GATE ? 8 : F32 ? 32 : 16;  // store instructions of a whole tile (vec)

    Lane c = lane_of();
    const int lda = p.K;
    const int tiles_n = (p.ncols + TNO - 1) / TNO;
    fill_table(tab, p, c);
    __syncthreads();
    zero_rows(p, 0, tab.first[0]);
    zero_rows(p, tab.first[p.E], p.M);
    const int ntiles = count_tiles(tab, p.E, tiles_n);
    const int nwg = gridDim.x, self = first_tile();
    if (self >= ntiles) return;
    // at least three stages (the surplus reads zeros): the next tile's row
    // indices and scales land within a tile
    const int nk = max((p.K + kRowBytes - 1) / kRowBytes, 3);
    auto find = [&](int round) {
        return find_tile(tab, p.E, ntiles, tiles_n, TNO, snake(round, nwg, self),
                         [&](const auto *at, int id) { return group_of(at, p.E, id, c); });
    };

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
    turn_end<0>();
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
        parity ^= 1;
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // nothing is left to land in LDS
}

// 64-row tiles of 64 columns over a deep ring (see moe_tiles_64), for a few rows
// per group: the time is the reading of W.  8 waves (4 x 2) of 16 x 32; with the
// gate a wave's 32 rows of W are 16 gate rows and the 16 up rows that meet
// them.  A tile's row indices are loaded two tiles ahead, its scales as in
// i8_tiles, all into LDS: the loads of the ring are waited for by count, and a
// load into registers would end that.
constexpr int kDeep = 8, kDeepPart = 64 * kRowBytes, kDeepSlot = 2 * kDeepPart, kDeepWait = (kDeep - 2) * 2;

template <bool GATE, bool F32>
__global__ __launch_bounds__(512, 1) void i8_tiles_64(I8Gemm p)
{
    __shared__ __attribute__((aligned(1024))) uint8_t lds[kDeep * kDeepSlot];
    __shared__ Table<64> tab;
    __shared__ uint32_t rowbuf[2][64];
    __shared__ __attribute__((aligned(16))) float scales[2][2][64];    // [parity of the tile][0: rows, 1: rows of W]
    constexpr int TNO = GATE ? 32 : 64, SZ = F32 ? 4 : 2;

    const Lane c = lane_of();
    const int wm = c.w >> 1, wn = c.w & 1, j = c.lane & 15, g = c.lane >> 4;
    const int lda = p.K;
    const int tiles_n = (p.ncols + TNO - 1) / TNO;
    fill_table(tab, p, c);
    __syncthreads();
    zero_rows(p, 0, tab.first[0]);
    zero_rows(p, tab.first[p.E], p.M);
    const int ntiles = count_tiles(tab, p.E, tiles_n);
    const int nwg = gridDim.x;
    int tile = first_tile();
    if (tile >= ntiles) return;
    // at least as many stages as slots: the loads turn to the next tile behind a
    // barrier of this one, when the tile before's scales have been read
    const int nk = max((p.K + kRowBytes - 1) / kRowBytes, kDeep);
    auto find = [&](int id) {
        return find_tile(tab, p.E, ntiles, tiles_n, TNO, id,
                         [&](const auto *at, int n) { return group_of(at, p.E, n, c); });
    };

    // wave w loads rows 8 w .. of A and of W
    i32x4 ra, rb;
    const int lrow = 8 * c.w + (c.lane >> 3);
    int rot = 0;
    uint32_t aoff = 0, boff = 0;
    uint32_t kx = (uint32_t)(((c.lane & 7) ^ swz(lrow)) << 4);     // the lane's chunk of its row
    // (one wave, one load: the others' count of loads under way is one less, which waits for no fewer)
    auto fetch = [&](const RowTile &r, int place) {
        if (c.w != 0 || !p.rows) return;
        dma<4>(words_of(p.rows + r.m0, (uint32_t)max(min(r.mend - r.m0, 64), 0) * 4u),
               reinterpret_cast<uint8_t *>(rowbuf), place * 256, (uint32_t)c.lane * 4u);
    };
    auto aim = [&](const RowTile &r, int place) {
        if (r.blocks == 0) {
            ra = rb = words_of(nullptr, 0);
            return;
        }
        // (the walk along K starts elsewhere per tile, as in moe_tiles_64)
        rot = r.n0 / TNO % nk;
        const int64_t wbytes = (int64_t)p.N * p.K;
        const uint8_t *wg = p.W + r.g * wbytes;
        const int left = min(r.mend - r.m0, 64);
        const uint32_t have = p.rows ? (uint32_t)p.T : (uint32_t)left;
        const uint32_t row = p.rows ? rowbuf[place][lrow] : (uint32_t)lrow;
        ra = words_of(p.rows ? p.X : p.X + (int64_t)r.m0 * lda, have * (uint32_t)lda);
        aoff = lrow < left && row < have ? row * (uint32_t)lda : kRowOOB;
        if constexpr (GATE) {
            // rows 32 wn + 16 u + q of the slot: row n0 + 16 wn + q of matrix u
            const int f = r.n0 + (lrow >> 5) * 16 + (lrow & 15);
            rb = words_of(wg, (uint32_t)wbytes);
            boff = f < p.ncols ? (uint32_t)((((lrow >> 4) & 1) * p.ncols + f) * lda) : kRowOOB;
        } else {
            rb = words_of(wg + (int64_t)r.n0 * lda, (uint32_t)(min(p.N - r.n0, 64) * lda));
            boff = (uint32_t)(lrow * lda);
        }
        if (c.w == 0) {
            const uint32_t at = p.rows ? rowbuf[place][c.lane] : (uint32_t)c.lane;
            dma<4>(words_of(p.rows ? p.sX : p.sX + r.m0, have * 4u), reinterpret_cast<uint8_t *>(scales), place * 512,
                   at < have ? at * 4u : kRowOOB);
        } else if (c.w == 1) {
            const int at = GATE ? ((c.lane >> 4) & 1) * p.ncols + r.n0 + (c.lane >> 5) * 16 + (c.lane & 15) : r.n0 + c.lane;
            dma<4>(words_of(p.sW + (int64_t)r.g * p.N, (uint32_t)p.N * 4u), reinterpret_cast<uint8_t *>(scales),
                   place * 512 + 256, at < p.N ? (uint32_t)at * 4u : kRowOOB);
        }
    };
    auto load = [&](int slot, int ks) {
        ks += rot;
        ks -= ks >= nk ? nk : 0;
        const uint32_t dst = slot * kDeepSlot;
        const int kc = (int)kx + ks * kRowBytes;
        const bool in = kc < lda;
        dma<16>(ra, lds, dst + c.w * 1024, in ? aoff + kc : kRowOOB);
        dma<16>(rb, lds, dst + kDeepPart + c.w * 1024, in ? boff + kc : kRowOOB);
    };

    int parity = 0;
    RowTile cur = find(tile), next = find(tile + nwg);
    fetch(cur, 0);
    fetch(next, 1);
    turn_end<0>();
    aim(cur, 0);
#pragma unroll
    for (int f = 0; f < kDeep - 1; ++f) load(f, f);
    const int ar = 16 * wm + j;
    uint32_t fa = (uint32_t)(ar * kRowBytes + ((kgroup(g) ^ swz(ar)) << 4)), fb = kDeepPart + part_base<false>(c, wn);
    stage_barrier<kDeepWait>();

    int rs = 0;               // slot the next stage reads
    for (;;) {
        tile += nwg;
        // (this tile's row indices have been read: their place is the tile's after the next one)
        const RowTile after = find(tile + nwg);
        fetch(after, parity);
        i32x4 acc[2] = {};
        for (int s = 0; s < nk; ++s) {
            int ks = s + kDeep - 1;
            if (ks >= nk) {
                ks -= nk;
                if (ks == 0) aim(next, parity ^ 1);
            }
            asm volatile("" : "+v"(kx), "+v"(fa), "+v"(fb));
            const uint32_t so = (uint32_t)(rs * kDeepSlot);
            bf16x8 a[2], b[2][2];
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
                a[kk] = lds_read<bf16x8>(lds, (fa ^ (uint32_t)(kk << 6)) + so);
#pragma unroll
                for (int u = 0; u < 2; ++u) b[kk][u] = part_frag<false>(lds, fb + so, kk, 0, u);
            }
            load(rs == 0 ? kDeep - 1 : rs - 1, ks);
#pragma unroll
            for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                for (int u = 0; u < 2; ++u) acc[u] = MulI8::mul(b[kk][u], a[kk], acc[u]);
            stage_barrier<kDeepWait>();
            rs = rs + 1 == kDeep ? 0 : rs + 1;
        }
        // lane: row 16 wm + l % 16, four columns of each block
        const int r0 = cur.m0 + 16 * wm, left = __builtin_amdgcn_readfirstlane(max(0, min(16, cur.mend - r0)));
        const __amdgpu_buffer_rsrc_t rd =
            make_rsrc(p.D + (int64_t)r0 * p.ncols * SZ, (uint32_t)left * (uint32_t)p.ncols * (uint32_t)SZ);
        const float sx = scales[parity][0][ar];
        f32x4 h[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const f32x4 sw = *reinterpret_cast<const f32x4 *>(&scales[parity][1][32 * wn + 16 * u + 4 * g]);
#pragma unroll
            for (int q = 0; q < 4; ++q) h[u][q] = (float)acc[u][q] * sx * sw[q];
        }
#pragma unroll
        for (int u = 0; u < (GATE ? 1 : 2); ++u) {
            float v[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] = GATE ? gated(h[0][q], h[1][q]) : h[u][q];
            const int n = cur.n0 + (GATE ? 16 : 32) * wn + 16 * u + 4 * g;
            store_four<F32>(rd, v, n, p.ncols, (uint32_t)(j * p.ncols + n) * (uint32_t)SZ, p.vec);
        }
        if (next.blocks == 0) break;
        cur = next;
        next = after;
        parity ^= 1;
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // nothing is left to land in LDS
}

// At most as many workgroups as there can be tiles of tm rows and tno columns.
dim3 tile_grid(const I8Gemm &p, int tm, int tno, int cus)
{
    const int64_t most = ((int64_t)p.M / tm + (p.M < p.E ? p.M : p.E)) * ((p.ncols + tno - 1) / tno);
    return dim3((uint32_t)(most < cus ? most : cus));
}

}  // namespace

hipError_t launch_i8_tiles(const I8Gemm &p, int rows, int cus, hipStream_t stream)
{
    const dim3 block(512);
    if (rows == 64) {
        const dim3 grid = tile_grid(p, 64, p.gate ? 32 : 64, cus);
        if (p.gate) hipLaunchKernelGGL((i8_tiles_64<true, false>), grid, block, 0, stream, p);
        else if (p.f32) hipLaunchKernelGGL((i8_tiles_64<false, true>), grid, block, 0, stream, p);
        else hipLaunchKernelGGL((i8_tiles_64<false, false>), grid, block, 0, stream, p);
    } else {
        auto go = [&](auto tm) {
            constexpr int TM = decltype(tm)::value;
            const dim3 grid = tile_grid(p, TM, p.gate ? 128 : 256, cus);
            if (p.gate) hipLaunchKernelGGL((i8_tiles<TM, true, false>), grid, block, 0, stream, p);
            else if (p.f32) hipLaunchKernelGGL((i8_tiles<TM, false, true>), grid, block, 0, stream, p);
            else hipLaunchKernelGGL((i8_tiles<TM, false, false>), grid, block, 0, stream, p);
        };
        if (rows == 256) go(std::integral_constant<int, 256>{});
        else go(std::integral_constant<int, 128>{});
    }
    return hipGetLastError();
}

}  // namespace dbs
