// moe_gemm.hip -- gfx950 kernels of the experts' products (bf16, fp32 sums):
//
//   tiles   D[i, n]      = sum_k X[rows[i], k] W_g[n, k]      i in group g; W_g K-major (N x K)
//           D[i, n]      = sum_k X[rows[i], k] W_g[k, n]      W_g MN-major (K x N): the rows' gradient
//           D[i, f]      = silu(h[f]) h[F + f]                h = the first form's row, F = N / 2 (the gate)
//   dw      dW_g[n, k]   = sum_i dY[i, n] X[rows[i], k]       over the rows i of group g
//
// The groups' row offsets are read on the device: a workgroup turns them
// into a table of first tiles in LDS, so a router's output needs no copy to
// the host.  The stages, their swizzles and fragment reads are those of the
// BF16 GEMM (gemm_kernel.h); what differs is where rows come from.
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

namespace dbs {
namespace {

constexpr uint32_t kRowOOB = 0xFF000000u;        // + a row's bytes (at most 2^22) still lies past every resource

// TM x 256 output tiles of 8 waves (2 x 4), each TM / 2 x 64, over NS slots.
// AMN / BMN: the operand's slots hold K-rows (see Mn in gemm_kernel.h).
template <int TM_, int NS_, bool AMN_, bool BMN_>
struct Tile {
    static constexpr int TM = TM_, TN = 256, NS = NS_, WM = 2, WN = 4, NW = 8, kThreads = 512;
    static constexpr bool AMN = AMN_, BMN = BMN_;
    static constexpr int MB = TM / WM / 32, NB = TN / WN / 32;
    static constexpr int QA = TM / 8 / NW, QB = TN / 8 / NW;       // wave-loads per wave and stage
    static constexpr int kSlotA = TM * kRowBytes, kSlotB = TN * kRowBytes;
    static constexpr int kLdsA = 0, kLdsB = NS * kSlotA, kRing = NS * (kSlotA + kSlotB);
    static constexpr int KS = 64;                                  // K per stage
    static_assert(QA > 0 && MB > 0, "every wave loads and computes");
};

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

template <class S, int MBA = S::MB>
struct Frag2 {
    bf16x8 a[MBA], b[S::NB];
};

// K-major A: the two wave rows take the tile's blocks of 32 rows in turn
// (wave row wm: blocks wm, wm + 2, ...), so a tile whose group ends early
// leaves both with the same number of blocks, MBA, to compute.  Blocks of one
// wave lie 64 rows apart, where the swizzle repeats.
template <class S>
__device__ __forceinline__ bf16x8 read_a2(const uint8_t *lds, uint32_t fa, int kk, int i)
{
    if constexpr (S::AMN) return read_frag_mn<kBF16, S::TM>(lds, fa, 0, kk, i);
    else return lds_read<bf16x8>(lds, (fa ^ (uint32_t)(kk << 5)) + (uint32_t)(64 * kRowBytes * i));
}

// One k-step: the MFMAs of `cur` while k-step PH of the slot behind fa / fb
// is read into `nxt` (if RD); after MFMA i, issue(i).
template <class S, int MBA, int PH, bool RD, class ISSUE>
__device__ __forceinline__ void phase2(f32x16 (&acc)[MBA][S::NB], Frag2<S, MBA> &cur, Frag2<S, MBA> &nxt,
                                       const uint8_t *lds, uint32_t fa, uint32_t fb, ISSUE &&issue)
{
    if constexpr (RD) {
#pragma unroll
        for (int i = 0; i < MBA; ++i) nxt.a[i] = read_a2<S>(lds, fa, PH, i);
#pragma unroll
        for (int j = 0; j < S::NB; ++j) {
            if constexpr (S::BMN) nxt.b[j] = read_frag_mn<kBF16, S::TN>(lds, fb, 0, PH, j);
            else nxt.b[j] = read_frag<kBF16>(lds, fb, 0, PH, j);
        }
    }
    DBS_FENCE();
#pragma unroll
    for (int i = 0; i < MBA; ++i) {
#pragma unroll
        for (int j = 0; j < S::NB; ++j) {
            mma1<kBF16, 0>(acc[i][j], cur.a[i], 0u, cur.b[j], 0u);
            DBS_FENCE();
            issue(PH * MBA * S::NB + i * S::NB + j);
            DBS_FENCE();
        }
    }
}

// One stage of four k-steps out of the slot behind fa / fb.  On entry F1
// holds the previous stage's last k-step, whose MFMAs come first; piece q of
// the stage being loaded goes out after MFMA q.
template <class S, int MBA, class PIECE>
__device__ __forceinline__ void stage2(f32x16 (&acc)[MBA][S::NB], Frag2<S, MBA> &F0, Frag2<S, MBA> &F1,
                                       const uint8_t *lds, uint32_t fa, uint32_t fb, PIECE &&piece)
{
    auto issue = [&](int i) {
        if (i < S::QB) piece(i);
    };
    static_assert(S::QA <= S::QB && S::QB <= 4 * S::NB, "piece q loads A (q < QA) and B");
    phase2<S, MBA, 0, true>(acc, F1, F0, lds, fa, fb, issue);
    phase2<S, MBA, 1, true>(acc, F0, F1, lds, fa, fb, issue);
    phase2<S, MBA, 2, true>(acc, F1, F0, lds, fa, fb, issue);
    phase2<S, MBA, 3, true>(acc, F0, F1, lds, fa, fb, issue);
    stage_barrier<(S::NS - 2) * (S::QA + S::QB)>();
}

// LDS addresses of the lane's fragment reads: slot 0, block 0, k-step 0.
template <class S>
__device__ __forceinline__ uint32_t frag_a(const Lane &c)
{
    if constexpr (S::AMN) return mn_base<kBF16, S::TM>(c.lane, c.wm * (S::TM / S::WM), S::kLdsA);
    const int r = c.wm * 32 + c.lr;
    return (uint32_t)(S::kLdsA + r * kRowBytes + ((c.h ^ swz(r)) << 4));
}

template <class S>
__device__ __forceinline__ uint32_t frag_b(const Lane &c)
{
    if constexpr (S::BMN) return mn_base<kBF16, S::TN>(c.lane, c.wn * (S::TN / S::WN), S::kLdsB);
    const int r = c.wn * (S::TN / S::WN) + c.lr;
    return (uint32_t)(S::kLdsB + r * kRowBytes + ((c.h ^ swz(r)) << 4));
}

// ------------------------------------------------------------ group tables

// first[g] = first row of group g (g <= E; offsets clamped to 0 .. M and made
// ascending; with FIRST), and at[g] = units of work before group g, per(rows)
// of them in a group: by one wave, the others wait at the caller's barrier.
template <bool FIRST, class T, class PER>
__device__ __forceinline__ void group_table(int32_t *first, T *at, const int32_t *offsets, int E, int M, const Lane &c,
                                            PER &&per)
{
    int hi = 0, sum = 0;                       // last row and work before this chunk of 64 groups
    if (c.lane == 0) {
        hi = min(max(offsets[0], 0), M);
        if constexpr (FIRST) first[0] = hi;
        at[0] = 0;
    }
    hi = __shfl(hi, 0);
    for (int g0 = 0; g0 < E; g0 += 64) {
        const int g = g0 + c.lane;
        int end = g < E ? min(max(offsets[g + 1], 0), M) : 0;
        end = max(end, hi);
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const int o = __shfl_up(end, d);
            if (c.lane >= d) end = max(end, o);
        }
        const int prev = __shfl_up(end, 1);
        const int rows = end - (c.lane == 0 ? hi : prev);
        int n = g < E ? per(rows) : 0;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const int o = __shfl_up(n, d);
            if (c.lane >= d) n += o;
        }
        if (g < E) {
            if constexpr (FIRST) first[g + 1] = end;
            at[g + 1] = (T)(sum + n);
        }
        hi = __shfl(end, 63);
        sum += __shfl(n, 63);
    }
}

// The last group g with at[g] <= id (groups without work have equal
// neighbours): 64 entries a step, one LDS read each.
template <class T>
__device__ __forceinline__ int group_of(const T *at, int E, int id, const Lane &c)
{
    int n = 0;
    for (int g0 = 0; g0 < E; g0 += 64) {
        const int g = g0 + c.lane;
        n += __popcll(__ballot(g < E && (int)at[g] <= id));
    }
    return __builtin_amdgcn_readfirstlane(n - 1);
}

__device__ __forceinline__ int first_tile()
{
    // workgroup w runs on XCD w % 8: every XCD takes a run of tiles
    const int nwg = gridDim.x, wg = blockIdx.x;
    return (nwg & 7) == 0 ? (wg & 7) * (nwg >> 3) + (wg >> 3) : wg;
}

// ---------------------------------------------------------------- epilogue

// The wave's accumulators as rows m0 .. mend-1, columns n0 .. ncols-1 of D
// (ld elements a row, OUT a bf16 or float): NBO blocks of 32 columns, value
// q of block j in block-row i from value(i, j, q).  vec: through LDS and in
// 16-byte pieces (bf16; the caller's slot is free); otherwise by element.
template <class S, int MBA, int NBO, class VALUE>
__device__ __forceinline__ void store_bf16(uint8_t *buf, uint8_t *D, int64_t ld, int m0, int mend, int n0, int ncols,
                                           int vec, Lane c, VALUE &&value)
{
    // (addresses are made here, not before the tile's stages, whose registers they would take)
    asm volatile("" : "+v"(c.lane), "+v"(c.lr), "+v"(c.h));
    constexpr int RB = NBO * 64, CPR = RB / 16, RPI = 64 / CPR;
#pragma unroll
    for (int i = 0; i < MBA; ++i) {
        const int r0 = m0 + (S::AMN ? c.wm * (S::TM / S::WM) + i * 32 : (2 * i + c.wm) * 32);
        const int left = __builtin_amdgcn_readfirstlane(max(0, min(32, mend - r0)));
        const __amdgpu_buffer_rsrc_t rd = make_rsrc(D + (int64_t)r0 * ld * 2, (uint32_t)left * (uint32_t)ld * 2u);
        if (vec) {
#pragma unroll
            for (int j = 0; j < NBO; ++j) {
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const uint32_t lo = pack_bf16(value(i, j, 4 * g), value(i, j, 4 * g + 1));
                    const uint32_t hi = pack_bf16(value(i, j, 4 * g + 2), value(i, j, 4 * g + 3));
                    const int ch = (4 * j + g) ^ (c.lr & (CPR - 1));
                    *reinterpret_cast<u32x2 *>(buf + c.lr * RB + 16 * ch + 8 * c.h) = u32x2{lo, hi};
                }
            }
#pragma unroll
            for (int q = 0; q < 32 / RPI; ++q) {
                const int r = q * RPI + c.lane / CPR, ch = c.lane % CPR;
                const i32x4 v = *reinterpret_cast<const i32x4 *>(buf + r * RB + 16 * (ch ^ (r & (CPR - 1))));
                const int n = n0 + ch * 8;
                __builtin_amdgcn_raw_buffer_store_b128(v, rd, n < ncols ? (uint32_t)(r * (int)ld + n) * 2u : kOOB, 0,
                                                       kStoreNT);
            }
        } else {
#pragma unroll
            for (int j = 0; j < NBO; ++j) {
#pragma unroll
                for (int q = 0; q < 16; ++q) {
                    const int n = n0 + j * 32 + (q / 4) * 8 + c.h * 4 + q % 4;
                    __builtin_amdgcn_raw_buffer_store_b16((uint16_t)pack_bf16(value(i, j, q), 0.0f), rd,
                                                          n < ncols ? (uint32_t)(c.lr * (int)ld + n) * 2u : kOOB, 0,
                                                          kStoreNT);
                }
            }
        }
    }
}

// ------------------------------------------------------------------- tiles

// A group of r rows has r / TM whole tile rows and a rest, computed with the
// ceil(rest / 64) blocks per wave that hold it.  Tiles are handed out by
// descending cost -- all groups' whole tile rows (and rests that need every
// block), then the rests by blocks -- in a snake over the workgroups, so
// that those with a tile less of one kind come first for the next.
template <class S>
struct Table {
    int32_t first[kMoeMaxExperts + 1], whole[kMoeMaxExperts + 1];   // tile rows before a group
    uint16_t rest[S::MB > 1 ? S::MB - 1 : 1][kMoeMaxExperts + 1];   // rests of b + 1 blocks before a group
};

// blocks per wave of a group's rest; S::MB counts as a whole tile row
template <class S>
__device__ __forceinline__ int rest_blocks(int rows) { return (rows % S::TM + 63) / 64; }

// GATE: see the head of the file.
template <class S, bool GATE>
__global__ __launch_bounds__(512, 1) void moe_tiles(MoeGemm p)
{
    __shared__ __attribute__((aligned(1024))) uint8_t lds[S::kRing];
    __shared__ Table<S> tab;
    static_assert(!(GATE && S::BMN), "the gate takes K-major matrices");
    constexpr int MB = S::MB, NB = S::NB;
    constexpr int TNO = GATE ? S::TN / 2 : S::TN;      // output columns of a tile

    const Lane c = lane_of();
    const int lda = p.K * 2;
    const int tiles_n = (p.ncols + TNO - 1) / TNO;
    if (c.w == 0)
        group_table<true>(tab.first, tab.whole, p.offsets, p.E, p.M, c,
                          [&](int rows) { return rows / S::TM + (rest_blocks<S>(rows) == MB); });
    else if (c.w < MB)
        group_table<false>(tab.first, tab.rest[c.w - 1], p.offsets, p.E, p.M, c,
                           [&](int rows) { return (int)(rest_blocks<S>(rows) == c.w); });
    __syncthreads();

    // rows behind the last group are zero
    {
        const int64_t total = tab.first[p.E];
        const int64_t bytes = (p.M - total) * p.ncols * 2;
        uint8_t *z = p.D + total * p.ncols * 2;
        const int64_t me = (int64_t)blockIdx.x * S::kThreads + threadIdx.x, all = (int64_t)gridDim.x * S::kThreads;
        if (p.vec)
            for (int64_t o = me * 16; o < bytes; o += all * 16) *reinterpret_cast<i32x4 *>(z + o) = i32x4{};
        else
            for (int64_t o = me * 2; o < bytes; o += all * 2) *reinterpret_cast<uint16_t *>(z + o) = 0;
    }

    int ntiles = __builtin_amdgcn_readfirstlane(tab.whole[p.E]);
#pragma unroll
    for (int b = 1; b < MB; ++b) ntiles += __builtin_amdgcn_readfirstlane((int)tab.rest[b - 1][p.E]);
    ntiles *= tiles_n;
    const int nwg = gridDim.x, self = first_tile();
    if (self >= ntiles) return;
    const int nk = max((p.K + S::KS - 1) / S::KS, S::NS - 1);

    struct Ref {
        int m0, mend, n0, g, blocks;
    };
    // output tile id of the order above; past the last: no rows
    auto ref_of = [&](int id) {
        Ref r{};
        if (id >= ntiles) return r;
        const int whole = __builtin_amdgcn_readfirstlane(tab.whole[p.E]) * tiles_n;
        if (id < whole) {
            const int row = id / tiles_n;              // groups of one tile row need no more than this
            r.g = group_of(tab.whole, p.E, row, c);
            const int before = __builtin_amdgcn_readfirstlane(tab.whole[r.g]);
            const int n = __builtin_amdgcn_readfirstlane(tab.whole[r.g + 1]) - before;
            const int local = id - before * tiles_n;   // tile rows fastest: they share W's rows
            r.m0 = local % n * S::TM;
            r.n0 = local / n * TNO;
            r.blocks = MB;
        } else {
            id -= whole;
#pragma unroll
            for (int b = MB - 1; b >= 1; --b) {
                const int n = __builtin_amdgcn_readfirstlane((int)tab.rest[b - 1][p.E]) * tiles_n;
                if (r.blocks == 0 && id < n) {
                    r.g = group_of(tab.rest[b - 1], p.E, id / tiles_n, c);
                    r.n0 = id % tiles_n * TNO;
                    r.blocks = b;
                }
                id -= r.blocks == 0 ? n : 0;
            }
        }
        const int lo = __builtin_amdgcn_readfirstlane(tab.first[r.g]);
        r.mend = __builtin_amdgcn_readfirstlane(tab.first[r.g + 1]);
        if (r.blocks < MB) r.m0 = (r.mend - lo) / S::TM * S::TM;
        r.m0 += lo;
        return r;
    };

    // where a tile's stages come from
    struct Source {
        __amdgpu_buffer_rsrc_t ra, rb;
        uint32_t a[S::QA];       // the lane's byte offset in ra per wave-load, its chunk included
        int f0;                  // the tile's first output column
    } src;
    // the rows of X behind the next tile's wave-loads, read while this tile is
    // computed (~0: none, a zero row)
    uint32_t row[S::QA];
    uint32_t x4 = (uint32_t)(((c.lane & 7) ^ (c.lane >> 3)) << 4);
    const int ldb = S::BMN ? p.N * 2 : lda;            // bytes of a row of W as stored
    uint32_t r8ldb = (uint32_t)((c.lane >> 3) * ldb);
    uint32_t mb[2] = {};
    if constexpr (S::BMN) {
        mb[0] = mn_dma_lane<kBF16, S::TN>(c.lane, 0, ldb);
        mb[1] = mn_dma_lane<kBF16, S::TN>(c.lane, 1, ldb);
    }
    auto fetch = [&](const Ref &r) {
#pragma unroll
        for (int q = 0; q < S::QA; ++q) {
            const int m = (c.w * S::QA + q) * 8 + (c.lane >> 3);
            row[q] = !p.rows ? (uint32_t)m : r.m0 + m < r.mend ? (uint32_t)p.rows[r.m0 + m] : ~0u;
        }
    };
    auto aim = [&](const Ref &r) {
        if (r.blocks == 0) {
            src.ra = src.rb = make_rsrc(nullptr, 0);
            return;
        }
        const int64_t wbytes = (int64_t)p.N * p.K * 2;
        const uint8_t *wg = p.W + r.g * wbytes;
        src.f0 = r.n0;
        if constexpr (S::BMN)
            src.rb = make_rsrc(wg + r.n0 * 2, (uint32_t)(wbytes - r.n0 * 2));
        else if constexpr (GATE)
            src.rb = make_rsrc(wg, (uint32_t)wbytes);
        else
            src.rb = make_rsrc(wg + (int64_t)r.n0 * lda, (uint32_t)(min(p.N - r.n0, S::TN) * lda));
        const uint32_t have = p.rows ? (uint32_t)p.T : (uint32_t)min(r.mend - r.m0, S::TM);
        src.ra = make_rsrc(p.rows ? p.X : p.X + (int64_t)r.m0 * lda, have * (uint32_t)lda);
#pragma unroll
        for (int q = 0; q < S::QA; ++q) {
            const int L = c.w * S::QA + q;
            src.a[q] = (row[q] < have ? row[q] * (uint32_t)lda : kRowOOB) + (x4 ^ (uint32_t)((L & 7) << 4));
        }
    };
    auto load = [&](int slot, int ks, int q) {
        const int k0 = ks * kRowBytes;
        if (q < S::QA) {
            const int L = c.w * S::QA + q;
            const int kc = (int)(x4 ^ (uint32_t)((L & 7) << 4));
            lds_dma<16>(src.ra, lds + S::kLdsA + slot * S::kSlotA + L * 1024, kc < lda - k0 ? src.a[q] + k0 : kRowOOB);
        }
        const int L = c.w * S::QB + q;
        uint8_t *dst = lds + S::kLdsB + slot * S::kSlotB + L * 1024;
        if constexpr (S::BMN) {
            const uint32_t row = (uint32_t)(ks * S::KS + L * 2);           // two K-rows a wave-load
            lds_dma<16>(src.rb, dst, row < (uint32_t)p.K ? mb[q & 1] + row * (uint32_t)ldb : kOOB);
        } else {
            const int kc = (int)(x4 ^ (uint32_t)((L & 7) << 4));
            uint32_t off = r8ldb + (uint32_t)(kc + k0);
            bool in = kc < lda - k0;
            if constexpr (GATE) {
                // rows 64 wn + 32 j + c of the slot: row f0 + 32 wn + c of matrix j
                const int r0 = L * 8, f = src.f0 + (r0 >> 6) * 32 + (r0 & 31);
                off += (uint32_t)((((r0 >> 5) & 1) * p.ncols + f) * lda);
                in = in && f + (c.lane >> 3) < p.ncols;
            } else {
                off += (uint32_t)(L * 8 * lda);
            }
            lds_dma<16>(src.rb, dst, in ? off : kOOB);
        }
    };

    Ref cur = ref_of(self), next{};
    fetch(cur);
    aim(cur);
#pragma unroll
    for (int f = 0; f < S::NS - 1; ++f) {
#pragma unroll
        for (int q = 0; q < S::QB; ++q) load(f, f, q);
    }
    uint32_t fa = frag_a<S>(c), fb = frag_b<S>(c);
    __syncthreads();

    int rs = 0;               // slot the next stage reads
    int round = 0;
    // one output tile of MBA blocks per wave
    auto run = [&](auto blocks) {
        constexpr int MBA = decltype(blocks)::value;
        f32x16 acc[MBA][NB];
#pragma unroll
        for (int i = 0; i < MBA; ++i)
#pragma unroll
            for (int j = 0; j < NB; ++j) acc[i][j] = f32x16{};
        Frag2<S, MBA> F0, F1{};
        int xs = 0;           // slot the last stage read
        for (int s = 0; s < nk; ++s) {
            int ks = s + S::NS - 1;
            if (ks >= nk) {
                ks -= nk;
                if (ks == 0) aim(next);
            }
            const int ls = rs == 0 ? S::NS - 1 : rs - 1;
            asm volatile("" : "+v"(x4), "+v"(r8ldb), "+v"(fa), "+v"(fb));
            stage2<S, MBA>(acc, F0, F1, lds, fa + (uint32_t)(rs * S::kSlotA), fb + (uint32_t)(rs * S::kSlotB),
                           [&](int q) { load(ls, ks, q); });
            xs = rs;
            rs = rs + 1 == S::NS ? 0 : rs + 1;
        }
        phase2<S, MBA, 0, false>(acc, F1, F0, lds, fa, fb, [](int) {});

        // the slot the last stage read is free until the next tile's first
        // stage refills it: its B part holds 8 waves' 32-row buffers
        constexpr int NBO = GATE ? NB / 2 : NB;
        uint8_t *buf = lds + S::kLdsB + xs * S::kSlotB + c.w * (32 * NBO * 64);
        store_bf16<S, MBA, NBO>(buf, p.D, p.ncols, cur.m0, cur.mend, cur.n0 + c.wn * (NBO * 32), p.ncols, p.vec, c,
                                [&](int i, int j, int q) {
                                    if constexpr (GATE) {
                                        const float g = acc[i][0][q];
                                        return g * __builtin_amdgcn_rcpf(1.0f + __expf(-g)) * acc[i][1][q];
                                    } else {
                                        return acc[i][j][q];
                                    }
                                });
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    };
    for (;;) {
        // the next tile's rows are looked up while this one is computed
        ++round;
        next = ref_of(round * nwg + (round & 1 ? nwg - 1 - self : self));
        fetch(next);
        if (MB == 1 || cur.blocks == MB) run(std::integral_constant<int, MB>{});
        if constexpr (MB > 1) {
            if (cur.blocks == 1) run(std::integral_constant<int, 1>{});
        }
        if constexpr (MB > 2) {
            if (cur.blocks == 2) run(std::integral_constant<int, 2>{});
            if (cur.blocks == 3) run(std::integral_constant<int, 3>{});
        }
        if (next.blocks == 0) break;
        cur = next;
    }
}

// ---------------------------------------------------------------------- dw

using DwTile = Tile<256, 2, true, true>;

// GATHER: rows of X through p.rows.  F32: dW holds fp32.
template <bool GATHER, bool F32>
__global__ __launch_bounds__(512, 1) void moe_dw(MoeGemmDw p)
{
    using S = DwTile;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[S::kRing];
    __shared__ int32_t first[kMoeMaxExperts + 1], tile_at[kMoeMaxExperts + 1];
    constexpr int MB = S::MB, NB = S::NB;

    const Lane c = lane_of();
    const int lda = p.N * 2, ldb = p.K * 2;            // bytes of a row of dY, of X
    const int tiles_n = (p.N + S::TM - 1) / S::TM, tiles_k = (p.K + S::TN - 1) / S::TN, per = tiles_n * tiles_k;
    if (c.w == 0)
        group_table<true>(first, tile_at, p.offsets, p.E, p.M, c,
                          [&](int rows) { return p.accumulate && rows == 0 ? 0 : per; });
    __syncthreads();
    const int ntiles = tile_at[p.E], nwg = gridDim.x;
    int tile = first_tile();
    if (tile >= ntiles) return;

    uint32_t ma[2] = {mn_dma_lane<kBF16, S::TM>(c.lane, 0, lda), mn_dma_lane<kBF16, S::TM>(c.lane, 1, lda)};
    // the lane's bytes within a K-row of X (gathered: the row's own offset is added)
    uint32_t mb[2] = {mn_dma_lane<kBF16, S::TN>(c.lane, 0, GATHER ? 0 : ldb),
                      mn_dma_lane<kBF16, S::TN>(c.lane, 1, GATHER ? 0 : ldb)};

    struct Ref {
        int lo, hi, n0, k0, g;
    };
    auto ref_of = [&](int id) {
        Ref r;
        r.g = group_of(tile_at, p.E, id, c);
        r.lo = __builtin_amdgcn_readfirstlane(first[r.g]);
        r.hi = __builtin_amdgcn_readfirstlane(first[r.g + 1]);
        const int local = id - __builtin_amdgcn_readfirstlane(tile_at[r.g]);
        r.n0 = local % tiles_n * S::TM;
        r.k0 = local / tiles_n * S::TN;
        return r;
    };
    auto stages = [](const Ref &r) { return max(1, (r.hi - r.lo + S::KS - 1) / S::KS); };
    Ref src{};                                         // the tile whose stages are loaded (hi = lo: nothing)
    const __amdgpu_buffer_rsrc_t rrows = make_rsrc(p.rows, GATHER ? (uint32_t)p.M * 4u : 0u);
    uint32_t idx[S::QB] = {};                          // X's rows of the lane's wave-loads in the next stage to load
    auto fetch_rows = [&](int ks) {
        if constexpr (GATHER) {
#pragma unroll
            for (int q = 0; q < S::QB; ++q) {
                const int m = src.lo + ks * S::KS + (c.w * S::QB + q) * 2 + c.h;
                idx[q] = m < src.hi ? __builtin_amdgcn_raw_buffer_load_b32(rrows, (uint32_t)m * 4u, 0, 0) : ~0u;
            }
        }
    };
    auto load = [&](int slot, int ks, int q) {
        const int m0 = src.lo + ks * S::KS, left = min(S::KS, src.hi - m0);       // rows of the stage
        const int L = c.w * S::QA + q;
        const uint32_t row = (uint32_t)(L * 2);
        const __amdgpu_buffer_rsrc_t ra =
            make_rsrc(p.dY + (int64_t)m0 * lda + src.n0 * 2, left > 0 ? (uint32_t)left * (uint32_t)lda - src.n0 * 2 : 0u);
        lds_dma<16>(ra, lds + S::kLdsA + slot * S::kSlotA + L * 1024, ma[q & 1] + row * (uint32_t)lda);
        uint8_t *dst = lds + S::kLdsB + slot * S::kSlotB + L * 1024;
        if constexpr (GATHER) {
            const __amdgpu_buffer_rsrc_t rb = make_rsrc(p.X + src.k0 * 2, (uint32_t)(p.T * ldb - src.k0 * 2));
            lds_dma<16>(rb, dst, idx[q] < (uint32_t)p.T ? idx[q] * (uint32_t)ldb + mb[q & 1] : kRowOOB);
        } else {
            const __amdgpu_buffer_rsrc_t rb = make_rsrc(p.X + (int64_t)m0 * ldb + src.k0 * 2,
                                                        left > 0 ? (uint32_t)left * (uint32_t)ldb - src.k0 * 2 : 0u);
            lds_dma<16>(rb, dst, mb[q & 1] + row * (uint32_t)ldb);
        }
    };

    Ref cur = ref_of(tile);
    src = cur;
    fetch_rows(0);
#pragma unroll
    for (int q = 0; q < S::QB; ++q) load(0, 0, q);
    int nk = stages(cur);
    uint32_t fa = frag_a<S>(c), fb = frag_b<S>(c);
    int next = tile + nwg;
    // rows of the stage after the first: this tile's, or the next tile's
    Ref nref = next < ntiles ? ref_of(next) : Ref{};
    if (nk > 1) {
        fetch_rows(1);
    } else {
        src = nref;
        fetch_rows(0);
    }
    __syncthreads();

    int rs = 0;
    for (;;) {
        f32x16 acc[MB][NB];
#pragma unroll
        for (int i = 0; i < MB; ++i)
#pragma unroll
            for (int j = 0; j < NB; ++j) acc[i][j] = f32x16{};
        Frag2<S> F0, F1{};
        for (int s = 0; s < nk; ++s) {
            // stage s + 1 of this tile, or the next tile's first, is loaded now; src and idx are its
            const int ks = s + 1 < nk ? s + 1 : 0;
            asm volatile("" : "+v"(ma[0]), "+v"(ma[1]), "+v"(mb[0]), "+v"(mb[1]), "+v"(fa), "+v"(fb));
            const int ls = rs ^ 1;
            auto issue = [&](int i) {
                if (i < S::QB) load(ls, ks, i);
            };
            const uint32_t a = fa + (uint32_t)(rs * S::kSlotA), b = fb + (uint32_t)(rs * S::kSlotB);
            phase2<S, MB, 0, true>(acc, F1, F0, lds, a, b, issue);
            // the row indices of the stage after that
            if (s + 2 < nk) {
                fetch_rows(s + 2);
            } else if (s + 2 == nk) {
                src = nref;
                fetch_rows(0);
            } else if (stages(nref) > 1) {
                fetch_rows(1);
            }
            phase2<S, MB, 1, true>(acc, F0, F1, lds, a, b, [](int) {});
            phase2<S, MB, 2, true>(acc, F1, F0, lds, a, b, [](int) {});
            phase2<S, MB, 3, true>(acc, F0, F1, lds, a, b, [](int) {});
            stage_barrier<0>();
            rs ^= 1;
        }
        phase2<S, MB, 0, false>(acc, F1, F0, lds, fa, fb, [](int) {});

        const int n0 = cur.n0, k0 = cur.k0 + c.wn * 64;
        if constexpr (F32) {
            // four consecutive columns a lane and block of four registers
            uint8_t *D = p.dW + (int64_t)cur.g * p.N * p.K * 4;
#pragma unroll
            for (int i = 0; i < MB; ++i) {
                const int r0 = n0 + c.wm * 128 + i * 32;
                const uint32_t left = __builtin_amdgcn_readfirstlane(max(0, min(32, p.N - r0)));
                const __amdgpu_buffer_rsrc_t rd = make_rsrc(D + (int64_t)r0 * p.K * 4, left * (uint32_t)p.K * 4u);
#pragma unroll
                for (int j = 0; j < NB; ++j) {
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        typedef __attribute__((ext_vector_type(4))) float f32x4;
                        const int k = k0 + j * 32 + g * 8 + c.h * 4;
                        const uint32_t off = k < p.K ? (uint32_t)(c.lr * p.K + k) * 4u : kOOB;   // K % 8 == 0
                        f32x4 v = {acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]};
                        if (p.accumulate)
                            v += __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(rd, off, 0, 0));
                        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(i32x4, v), rd, off, 0, kStoreNT);
                    }
                }
            }
        } else {
            uint8_t *buf = lds + S::kLdsB + (rs ^ 1) * S::kSlotB + c.w * (32 * NB * 64);
            store_bf16<S, MB, NB>(buf, p.dW + (int64_t)cur.g * p.N * p.K * 2, p.K, n0, p.N, k0, p.K, 1, c,
                              [&](int i, int j, int q) { return acc[i][j][q]; });
        }
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        if (next >= ntiles) break;
        tile = next;
        cur = nref;
        nk = stages(cur);
        next = tile + nwg;
        nref = next < ntiles ? ref_of(next) : Ref{};
        // a tile of one stage: the stage after it is the next tile's first
        if (nk == 1) {
            src = nref;
            fetch_rows(0);
        }
    }
}

template <class S>
hipError_t launch_tiles(const MoeGemm &p, int cus, hipStream_t stream)
{
    const int tno = p.gate ? S::TN / 2 : S::TN;
    const int64_t most = ((int64_t)p.M / S::TM + (p.M < p.E ? p.M : p.E)) * ((p.ncols + tno - 1) / tno);
    const dim3 grid((uint32_t)(most < cus ? (most > 0 ? most : 1) : cus));
    if constexpr (!S::BMN) {
        if (p.gate) {
            hipLaunchKernelGGL((moe_tiles<S, true>), grid, dim3(S::kThreads), 0, stream, p);
            return hipGetLastError();
        }
    }
    hipLaunchKernelGGL((moe_tiles<S, false>), grid, dim3(S::kThreads), 0, stream, p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_moe_tiles(const MoeGemm &p, int tm, int cus, hipStream_t stream)
{
    if (p.wmn) {
        switch (tm) {
        case 64: return launch_tiles<Tile<64, 3, false, true>>(p, cus, stream);
        case 128: return launch_tiles<Tile<128, 3, false, true>>(p, cus, stream);
        case 256: return launch_tiles<Tile<256, 2, false, true>>(p, cus, stream);
        }
    } else {
        switch (tm) {
        case 64: return launch_tiles<Tile<64, 3, false, false>>(p, cus, stream);
        case 128: return launch_tiles<Tile<128, 3, false, false>>(p, cus, stream);
        case 256: return launch_tiles<Tile<256, 2, false, false>>(p, cus, stream);
        }
    }
    return hipErrorInvalidValue;
}

hipError_t launch_moe_dw(const MoeGemmDw &p, int cus, hipStream_t stream)
{
    const int64_t tiles = (int64_t)p.E * ((p.N + 255) / 256) * ((p.K + 255) / 256);
    const dim3 grid((uint32_t)(tiles < cus ? tiles : cus)), block(DwTile::kThreads);
    if (p.rows) {
        if (p.f32) hipLaunchKernelGGL((moe_dw<true, true>), grid, block, 0, stream, p);
        else hipLaunchKernelGGL((moe_dw<true, false>), grid, block, 0, stream, p);
    } else {
        if (p.f32) hipLaunchKernelGGL((moe_dw<false, true>), grid, block, 0, stream, p);
        else hipLaunchKernelGGL((moe_dw<false, false>), grid, block, 0, stream, p);
    }
    return hipGetLastError();
}

}  // namespace dbs
