// moe_tiles.h -- index arithmetic of the experts' products: the order in which
// output tiles are handed out and the swizzles of their LDS parts.  Compiled
// for the device by moe_gemm.hip and for the host by the tests.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe.h"

#define DBS_BOTH __host__ __device__ __forceinline__

namespace dbs {

// A value that is the same in every lane, as a scalar
DBS_BOTH int same(int v)
{
#if defined(__HIP_DEVICE_COMPILE__)
    return __builtin_amdgcn_readfirstlane(v);
#else
    return v;
#endif
}

// ----------------------------------------------------------------- swizzles

// The eight K of a 32-deep step that lanes 16 g .. 16 g + 15 hold (see the math
// of the core).
DBS_BOTH constexpr int kgroup(int g) { return (g >> 1) | (g & 1) << 1; }

// MN-major swizzle of K-row r, in 16-byte chunks: the transposed reads of 32
// lanes take 32 bytes of four K-rows of two groups, 8 or 16 K-rows apart: rows
// 1 apart move by 64 bytes, rows 8 or 16 apart by 32.
DBS_BOTH constexpr int mn_swz(int r) { return 4 * (r & 3) ^ 2 * (((r >> 3) ^ (r >> 4)) & 1); }

// The same for 64 columns a K-row (dY in the small tiles of dW): the reads of
// two groups take 32 bytes of four K-rows each, and two K-rows share a bank line.
DBS_BOTH constexpr int narrow_swz(int r) { return 2 * ((r >> 1) & 1) ^ 4 * (((r >> 3) ^ (r >> 4)) & 1); }

// ----------------------------------------------------------- order of tiles

// The tile of a workgroup's turn `round`: a snake over the nwg workgroups.
DBS_BOTH int snake(int round, int nwg, int self) { return round * nwg + (round & 1 ? nwg - 1 - self : self); }

// A group of r rows has r / TM whole tile rows and a rest, computed with the
// ceil(rest / 64) blocks per wave that hold it.  Tiles are handed out by
// descending cost -- all groups' whole tile rows (and rests that need every
// block), then the rests by blocks -- in a snake over the workgroups, so
// that those with a tile less of one kind come first for the next.
template <int TM>
struct Table {
    static constexpr int kRests = TM / 64 - 1;
    // blocks of a group's rest; whole tile rows (and rests that need every block); whether it has a rest of b
    static DBS_BOTH int blocks(int rows) { return (rows % TM + 63) / 64; }
    static DBS_BOTH int whole_of(int rows) { return rows / TM + (blocks(rows) == TM / 64); }
    static DBS_BOTH int rest_of(int rows, int b) { return blocks(rows) == b; }

    int32_t first[kMoeMaxExperts + 1], whole[kMoeMaxExperts + 1];   // tile rows before a group
    uint16_t rest[kRests > 0 ? kRests : 1][kMoeMaxExperts + 1];     // rests of b + 1 blocks before a group
};

constexpr int kBand = 4;              // tile rows of a group handed out together

struct RowTile {
    int m0, mend, n0, g, blocks;      // blocks 0: nothing
};

template <int TM>
DBS_BOTH int count_tiles(const Table<TM> &tab, int E, int tiles_n)
{
    int n = same(tab.whole[E]);
#pragma unroll
    for (int b = 0; b < Table<TM>::kRests; ++b) n += same((int)tab.rest[b][E]);
    return n * tiles_n;
}

// Output tile id of the order above, tno columns wide.  group_of(at, id): the
// last group g with at[g] <= id.
template <int TM, class GROUP_OF>
DBS_BOTH RowTile find_tile(const Table<TM> &tab, int E, int ntiles, int tiles_n, int tno, int id, GROUP_OF &&group_of)
{
    constexpr int MB = TM / 64;
    RowTile r{};
    if (id >= ntiles) return r;
    const int whole = same(tab.whole[E]) * tiles_n;
    if (id < whole) {
        r.g = group_of(tab.whole, id / tiles_n);
        const int before = same(tab.whole[r.g]);
        const int n = same(tab.whole[r.g + 1]) - before;
        // bands of kBand tile rows, columns outside them: the tiles that one
        // XCD's workgroups hold together share rows of X and of W in its L2
        const int local = id - before * tiles_n, band = local / (kBand * tiles_n);
        const int rows = min(n - band * kBand, kBand), in = local - band * kBand * tiles_n;
        r.m0 = (band * kBand + in % rows) * TM;
        r.n0 = in / rows * tno;
        r.blocks = MB;
    } else {
        id -= whole;
#pragma unroll
        for (int b = MB - 1; b >= 1; --b) {
            const int n = same((int)tab.rest[b - 1][E]) * tiles_n;
            if (r.blocks == 0 && id < n) {
                r.g = group_of(tab.rest[b - 1], id / tiles_n);
                r.n0 = id % tiles_n * tno;
                r.blocks = b;
            }
            id -= r.blocks == 0 ? n : 0;
        }
    }
    const int lo = same(tab.first[r.g]);
    r.mend = same(tab.first[r.g + 1]);
    if (r.blocks < MB) r.m0 = (r.mend - lo) / TM * TM;
    r.m0 += lo;
    return r;
}

}  // namespace dbs
