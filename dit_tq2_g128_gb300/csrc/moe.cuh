// What the kernels of a mixture of experts share: sizes, the table of its work and the staged activations.
#pragma once

#include <algorithm>

#include "tq2_internal.cuh"

namespace tq2 {

// Some tokens of one expert: rows row0 .. row0 + n - 1 of those sorted by expert.
struct alignas(16) MoeTile {
    int expert, row0, n, unused;
};

// Device tables of one call, from its routing: `rows` (token, expert) pairs sorted by expert, and their tiles.
struct MoePlan {
    int *tile_count;      // [2]: tiles, rows
    MoeTile *tiles;
    int *pair_row;        // [pairs] row of each pair, -1: none
    int *expert_rows;     // [experts]
    float2 *bound;        // [experts][bound_blocks] of some of an expert's features (see below)
};

// One ternary product of the layer: of staged activations (see moe_stage_kernel) with the rows of each tile's expert.
struct MoeGemm {
    MoePlan plan;
    const uint8_t *qs;   // codes [experts * rows][k / 4]
    const __half *d;     // block scales [experts * rows][k / 128]
    const void *staged;  // binary16, or e4m3 where terms is 3
    const float *scale;  // of each row: what its staged values are to be multiplied by
    const float *sum;    // gate_up: of each row, the sum of |x|
    const float *peak;   //          and the largest of a block of 128
    float *out;          // [rows][features]: of down the product, of gate_up, with three terms, the hidden values
    __half *staged_out;  // gate_up, one or two terms: the hidden values, staged
    float *scale_out;    //          and each row's scale
    int64_t pairs;
    int experts, rows, k;
    int terms;           // staged rows of a row
    int cols;            // staged rows (MMA columns) of a tile, at most: 32, 64 or 96, or 48 with three terms
    int max_tiles, bound_blocks;
};
// gate_up: rows counts gate then up rows, and the SwiGLU of rows / 2 features is staged; else out is the product.
cudaError_t launch_moe_gemm(const MoeGemm &g, bool gate_up, const LaunchCtx &ctx);

// Terms of a staged value v, scaled by a power of two to below 2^15 (2^8 for e4m3):
//   1: binary16(v).   2: also binary16((v - first) 2^12), at most 2^15: what is left of v has 11 bits as long as v is 2^-14 or
//      more, 2^-29 of the most (as it is it would lose bits from 2^-2 on, below 2^-17 of the most).
//   3: e4m3 numbers t0, t1, t2 with v = t0 + t1 / 16 + t2 / 256: each rounds to four bits what is left, so that they hold
//      twelve: all of a binary16's or bf16's (down to 2^-25 of the largest value), and others to 2^-12.
// Three 8-bit terms where experts have few tokens: an MMA of few columns takes as long for 32 weights of a row in 8 bits as
// for 16 in 16 bits, and decoding to 8 bits is half the stores and no subtraction.  Measured against one binary16 term: see
// form_of in moe.cu (one token of 6 of 64 experts of 2048 x 1408: 19.3 against 18.9 us, a launch more).
//
// Scale of staged hidden values, which the first product stages before any of its row is known to all: a bound of them.
// |Gate_f x| and |Up_f x| are at most 2 (code 3) times the sum over blocks of |d| times the block's sum of |x|, so that
//   |h_f| <= (2 S)^2 P, P the largest over f of a product of a number of the gate row and one of the up row:
// with S the sum of |x| of the row, their largest |d|; with S that of the block where it is largest, their sums of |d|.  The
// smaller of both is taken (the second where few scales are large, the first where few elements are).  By a product over the
// same feature, a large gate row counts once.
//
// Order of staged activations: a binary16 row holds elements i and i + 8 of each group of 16 at 2 i and 2 i + 1, as pairs of
// codes are masked out of a word of 16 (the library's binary16 activation layout).  An e4m3 row holds the even and the odd elements
// of each 8 after each other, as codes are looked up from a word four at a time.
__host__ __device__ constexpr int moe_place(int i) { return i < 8 ? 2 * i : 2 * (i - 8) + 1; }
__host__ __device__ constexpr int moe_place8(int i) { return (i & 8) + (i & 1) * 4 + (i & 7) / 2; }

constexpr float kLowScale = 4096.f;  // of the second of two terms

// 2^e with e kept to what f32 holds as a normal number.
__device__ __forceinline__ float moe_power(int e) { return __uint_as_float(uint32_t(max(min(e, 127), -126) + 127) << 23); }
// log2 of a positive finite f32, downwards (below 2^-126: -127).
__device__ __forceinline__ int moe_log2(float x) { return int(__float_as_uint(x) >> 23) - 127; }

}  // namespace tq2
