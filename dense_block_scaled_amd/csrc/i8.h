// i8.h -- internal interface between the C ABI of the 8-bit integer operators
// (i8.cpp) and their gfx950 kernels (i8_gemm.hip, i8_quant.hip).  Not
// installed; callers use include/dbs.h.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dbs {

// Products of codes, summed as 32-bit integers, times a scale per row of X and one per row
// of W.  Dense: offsets and rows null, E = 1, T = M.  Otherwise group g
// owns rows offsets[g] .. offsets[g+1]-1 of the sorted order, as in MoeGemm.
struct I8Gemm {
    const uint8_t *X;         // T x K codes (gathered through rows) or M x K
    const uint8_t *W;         // E x N x K codes
    const float *sX;          // T
    const float *sW;          // E x N
    uint8_t *D;               // M x ncols, bf16 or fp32
    const int32_t *offsets;   // E + 1, or null
    const int32_t *rows;      // M, or null
    int64_t T;                // rows of X
    int M, E, N, K;
    int ncols;                // columns of D: N, or N / 2 behind the gate
    int ldd;                  // elements from one row of D to the next
    int gate;                 // 1: D = silu(first N/2 columns) * last N/2 columns
    int f32;                  // 1: D holds fp32 (without the gate)
    int vec;                  // 1 if D rows take 16-byte stores
};

// An output tile: 16 rows by 16 columns; 16 by the columns of 64 rows of W; 64 by those of 64, 32 or (without
// the gate) 16; 128 by those of 128 or 64; 256 by those of 256.
struct I8Tile {
    int rows, cols;
};
// The tile for M rows over E groups on `cus` compute units (the rule and what it
// rests on: i8.cpp)
I8Tile i8_tile(int64_t M, int64_t E, int64_t N, int64_t ncols, int64_t K, bool gate, int cus, double *us = nullptr);
// The dense product's first launch: all M rows and N columns, or fewer of one where a
// second one for the others pays
struct I8Part {
    int64_t rows, cols;
};
I8Part i8_part(int64_t M, int64_t N, int64_t K, int cus);
hipError_t launch_i8_tiles(const I8Gemm &p, I8Tile tile, int cus, hipStream_t stream);

// Row scales and codes of x (M x K, fp32 or bf16).
hipError_t launch_quant_i8(const void *x, int bf16, int64_t M, int64_t K, int8_t *codes, float *scales,
                           hipStream_t stream);

}  // namespace dbs

// For the tests that say which kernel a size reaches (not in include/dbs.h): 1000 rows + cols of the tile; the
// rows of the dense product's first launch, or -columns where it has all rows
extern "C" int dbs_i8_tile(int64_t M, int64_t E, int64_t N, int64_t K, int gate, int cus);
extern "C" int64_t dbs_i8_part(int64_t M, int64_t N, int64_t K, int cus);
