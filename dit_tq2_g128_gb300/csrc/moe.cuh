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
    int *counts;       // [2]: tiles, rows
    MoeTile *tiles;
    int *row_pair;     // [pairs] pair of each row
    int *pair_row;     // [pairs] row of each pair, -1: none
};

// One ternary product of the layer: of staged activations (see moe_stage_kernel) with the rows of each tile's expert.
struct MoeGemm {
    MoePlan plan;
    const uint8_t *qs;   // codes [experts * rows][k / 4]
    const __half *d;     // block scales [experts * rows][k / 128]
    const __half *staged;
    const float *scale;  // of each row
    float *out;          // [rows][features]
    int64_t pairs;
    int experts, rows, k;
    int terms;           // staged rows of a row
    int cols;            // staged rows (MMA columns) of a tile, at most: 64 or 128
    int max_tiles;
};
// gate_up: rows holds gate then up rows, out the SwiGLU of rows / 2 features; else out is the product.
cudaError_t launch_moe_gemm(const MoeGemm &g, bool gate_up, const LaunchCtx &ctx);

// Order of staged activations: a staged row holds elements i and i + 8 of each group of 16 at 2 i and 2 i + 1, as pairs of
// codes are masked out of a word of 16 (the library's binary16 activation layout).

}  // namespace tq2
