// Mixture of ternary experts:
//     out[t] = residual[t] + sum_j weight[t, j] Down_e (silu(Gate_e x_t) * (Up_e x_t)),  e = expert[t, j].
//
// The (token, expert) pairs are sorted by expert, so that an expert's codes are read once for all its tokens; each pair's
// activations are staged as terms that the tensor cores multiply (moe.cuh; moe_stage_kernel, which also sorts up to 1024
// pairs; more are sorted by moe_plan_kernel).  The first product (moe_gemm.cu) ends in the SwiGLU and stages its hidden values
// itself, scaled by a bound of them (moe.cuh); of few tokens it leaves them in f32, as e4m3 terms want the rows' largest
// values, and they are staged like the activations.  Each token's pairs of the second product are summed in their order
// (moe_sum_kernel): the same bits on every call.
//
// Bound by launches where tokens are few (one token of 6 experts: 19 us, five launches, of which the products are 10 + 8); of a
// prompt of 4096 tokens (531 us) staging writes 134 MB in 35 us, the sum reads 268 MB in 60 us (what the product before it
// wrote is still on its way to memory), the products are the rest.
#include <cstdint>

#include <cuda_fp8.h>

#include "cluster.cuh"
#include "dtype.cuh"
#include "moe.cuh"
#include "paged_attention.cuh"

namespace tq2 {
namespace {

constexpr int kPlanThreads = 1024, kPlanMaxCluster = 8, kPlanPairs = 4096;  // pairs of a CTA before there are more of them

// Exclusive sum over the block's threads (of WARPS warps) of v; total: the sum.
template <int WARPS>
__device__ __forceinline__ int block_scan(int v, int *part, int *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += x;
    }
    __syncthreads();
    if (lane == 31) part[warp] = s;
    __syncthreads();
    if (warp == 0) {
        int x = lane < WARPS ? part[lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        part[lane] = x;
    }
    __syncthreads();
    *total = part[31];
    return s - v + (warp ? part[warp - 1] : 0);
}

// The pairs sorted by expert, and the tiles.  One cluster, a part of the pairs a CTA.  (Counters place the pairs of one expert
// in whatever order they come; no result depends on it.)
__global__ void __launch_bounds__(kPlanThreads)
moe_plan_kernel(const int32_t *__restrict__ expert, MoePlan plan, int pairs, int experts, int tile_rows, int cluster,
                unsigned int *status) {
    __shared__ int count[1024], next[1024], part[32];
    const int tid = threadIdx.x, rank = int(cluster_rank());
    count[tid] = 0;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __syncthreads();
    const int per = (pairs + cluster - 1) / cluster, first = rank * per, last = min(pairs, first + per);
    bool bad = false;
    constexpr int U = 4;
    for (int p0 = first + tid; p0 < last; p0 += U * kPlanThreads) {
        int e[U];
#pragma unroll
        for (int i = 0; i < U; ++i) e[i] = p0 + i * kPlanThreads < last ? expert[p0 + i * kPlanThreads] : -1;
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (e[i] >= 0 && e[i] < experts)
                atomicAdd(&count[e[i]], 1);
            else
                bad |= e[i] != -1;
        }
    }
    report_bad(bad, status);
    cluster_sync();
    // thread e: expert e's rows, those of the CTAs before this one first
    int total = 0, before = 0;
    if (tid < experts)
        for (int c = 0; c < cluster; ++c) {
            const int n = at_cta(count, uint32_t(c))[tid];
            before += c < rank ? n : 0;
            total += n;
        }
    int rows, tiles;
    const int at = block_scan<kPlanThreads / 32>(total, part, &rows);
    const int n_tiles = (total + tile_rows - 1) / tile_rows;
    const int tile0 = block_scan<kPlanThreads / 32>(n_tiles, part, &tiles);
    next[tid] = at + before;
    if (rank == 0) {
        for (int i = 0; i < n_tiles; ++i)
            plan.tiles[tile0 + i] = MoeTile{tid, at + i * tile_rows, min(tile_rows, total - i * tile_rows), 0};
        if (tid < experts) plan.expert_rows[tid] = total;
        if (tid == 0) {
            plan.tile_count[0] = tiles;
            plan.tile_count[1] = rows;
        }
    }
    __syncthreads();
    for (int p0 = first + tid; p0 < last; p0 += U * kPlanThreads) {
        int e[U];
#pragma unroll
        for (int i = 0; i < U; ++i) e[i] = p0 + i * kPlanThreads < last ? expert[p0 + i * kPlanThreads] : -1;
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (p0 + i * kPlanThreads < last)
                plan.pair_row[p0 + i * kPlanThreads] = e[i] >= 0 && e[i] < experts ? min(atomicAdd(&next[e[i]], 1), pairs - 1) : -1;
    }
    cluster_sync();  // (the counts stay until all CTAs have read them)
}

constexpr int kStageThreads = 128;
constexpr int kFewPairs = 1024;     // that are sorted by the blocks that stage them
constexpr int kBoundScales = 1024;  // gate scales, and as many up scales, of a block that bounds an expert's hidden values

struct StageArgs {
    MoePlan plan;
    void *staged;    // [pairs][terms][k]
    float *scale;    // [pairs]
    float *sum;      // [pairs] of |x|, not below it
    float *peak;     // [pairs] the largest sum of |x| in a block of 128, not below it
    const __half *d;  // of gate and up
    int ffn;
    int bound_blocks, bound_rows, bound_lanes;  // of an expert; features of one; threads that share a feature
    int64_t tokens;
    int k, top_k, terms, experts;
    // where the pairs are not sorted yet
    const int32_t *expert;
    int tile_rows;
    unsigned int *status;
};

// Stages a token a block: the terms of its row times the power of two that brings its largest value between 2^14 and 2^15
// (no value overflows, and one 2^-28 of the largest still has all bits of a binary16; e4m3: between 2^7 and 2^8), in the products'
// order, to the rows of all its pairs; scale is the power that undoes it.  Of a row with an infinity or a NaN, e4m3 terms
// hold neither: its scale is NaN.  The blocks behind the tokens' bound some hidden values of an expert that has tokens (see
// moe.cuh).  PAIRS: the rows are of pairs already (hidden values).
// ROUTE: the pairs (at most kFewPairs) are not sorted yet: each token's block finds the rows of its pairs by counting those
// before them, and the first block behind the tokens' writes the tiles.
// At most 32 registers where tokens are few: beside a product's CTA an SM has 4096 left, so that blocks begin while the kernel
// before ends, and the next product's CTAs beside them (with 36, 7 tokens of 8 experts of 4096 x 6144 took 65 us, not 55).
template <typename T, bool F8, bool PAIRS, bool ROUTE>
__global__ void __launch_bounds__(kStageThreads, ROUTE || F8 ? 16 : 12) moe_stage_kernel(const T *__restrict__ x, const StageArgs a) {
    extern __shared__ uint4 bound_scales[];
    __shared__ float part[3][kStageThreads / 32];
    __shared__ int to[32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __shared__ int id[ROUTE ? kFewPairs : 1];
    const int pairs = ROUTE ? int(a.tokens) * a.top_k : 0;
    if constexpr (ROUTE) {
        for (int i = tid; i < pairs; i += kStageThreads) id[i] = a.expert[i];
    }
    if (!F8 && blockIdx.x >= a.tokens + ROUTE) {
        const int b = int(blockIdx.x - a.tokens - ROUTE), e = b / a.bound_blocks, f0 = b % a.bound_blocks * a.bound_rows;
        bool there = !ROUTE && a.plan.expert_rows[e] > 0;
        for (int i = tid; i < pairs; i += kStageThreads) there |= id[i] == e;  // (this thread's own)
        if (!__syncthreads_or(there)) return;
        // |d| of the features' gate rows, then of their up rows (features in multiples of 8: whole packs)
        const int nb = a.k / kBlockW, n = min(a.bound_rows, a.ffn - f0), packs = n * nb / 8;
        const uint4 *gate = reinterpret_cast<const uint4 *>(a.d + (int64_t(e) * 2 * a.ffn + f0) * nb);
        const uint4 *up = reinterpret_cast<const uint4 *>(a.d + (int64_t(e) * 2 * a.ffn + a.ffn + f0) * nb);
#pragma unroll 4
        for (int i = tid; i < 2 * packs; i += kStageThreads) {
            const uint4 v = i < packs ? gate[i] : up[i - packs];
            bound_scales[i] = make_uint4(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu, v.z & 0x7fff7fffu, v.w & 0x7fff7fffu);
        }
        __syncthreads();
        const __half *d = reinterpret_cast<const __half *>(bound_scales);
        float most = 0.f, whole = 0.f;  // of a feature's products: of its rows' largest scales, of their sums
        for (int f1 = 0; f1 < n; f1 += kStageThreads / a.bound_lanes) {
            const int f = f1 + tid / a.bound_lanes;
            float mg = 0.f, mu = 0.f, sg = 0.f, su = 0.f;
            if (f < n)
                for (int i = f * nb + tid % a.bound_lanes; i < (f + 1) * nb; i += a.bound_lanes) {
                    const float g = __half2float(d[i]), u = __half2float(d[8 * packs + i]);
                    mg = fmaxf(mg, g);
                    mu = fmaxf(mu, u);
                    sg += g;
                    su += u;
                }
            for (int o = a.bound_lanes / 2; o; o >>= 1) {
                mg = fmaxf(mg, __shfl_xor_sync(0xffffffffu, mg, o));
                mu = fmaxf(mu, __shfl_xor_sync(0xffffffffu, mu, o));
                sg += __shfl_xor_sync(0xffffffffu, sg, o);
                su += __shfl_xor_sync(0xffffffffu, su, o);
            }
            most = fmaxf(most, mg * mu);  // (a NaN is left out: all that its expert gives is NaN)
            whole = fmaxf(whole, sg * su);
        }
        most = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(most)));
        whole = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(whole)));
        if (lane == 0) {
            part[0][warp] = most;
            part[1][warp] = whole;
        }
        __syncthreads();
        if (tid == 0) {
            for (int w = 0; w < kStageThreads / 32; ++w) {
                most = fmaxf(most, part[0][w]);
                whole = fmaxf(whole, part[1][w]);
            }
            a.plan.bound[b] = make_float2(sqrtf(most), sqrtf(whole));
        }
        return;
    }
    if constexpr (ROUTE) {
        __shared__ int count[1024], sums[32];
        if (int64_t(blockIdx.x) == a.tokens) {
            for (int e = tid; e < 1024; e += kStageThreads) count[e] = 0;
            __syncthreads();
            for (int i = tid; i < pairs; i += kStageThreads) {
                const bool there = id[i] >= 0 && id[i] < a.experts;
                if (there) atomicAdd(&count[id[i]], 1);
                report_bad(!there && id[i] != -1, a.status);
            }
            __syncthreads();
            // experts 8 tid .. 8 tid + 7
            int rows = 0, tiles = 0;
            for (int e = 8 * tid; e < 8 * tid + 8; ++e) {
                rows += count[e];
                tiles += (count[e] + a.tile_rows - 1) / a.tile_rows;
            }
            int all_rows, all_tiles;
            int row = block_scan<kStageThreads / 32>(rows, sums, &all_rows), tile = block_scan<kStageThreads / 32>(tiles, sums, &all_tiles);
            for (int e = 8 * tid; e < 8 * tid + 8; ++e) {
                for (int i = 0; i < count[e]; i += a.tile_rows)
                    a.plan.tiles[tile++] = MoeTile{e, row + i, min(a.tile_rows, count[e] - i), 0};
                row += count[e];
            }
            if (tid == 0) {
                a.plan.tile_count[0] = all_tiles;
                a.plan.tile_count[1] = all_rows;
            }
            return;
        }
        if (tid < a.top_k) to[tid] = 0;
        __syncthreads();
        for (int j = 0; j < a.top_k; ++j) {
            const int p = int(blockIdx.x) * a.top_k + j, e = id[p];
            int before = 0;
            for (int i = tid; i < pairs; i += kStageThreads) before += id[i] >= 0 && (id[i] < e || (id[i] == e && i < p));
            before = __reduce_add_sync(0xffffffffu, before);
            if (lane == 0) atomicAdd(&to[j], before);
        }
        __syncthreads();
        if (tid < a.top_k) {
            const int p = int(blockIdx.x) * a.top_k + tid, e = id[p];
            if (e < 0 || e >= a.experts) to[tid] = -1;
            a.plan.pair_row[p] = to[tid];
        }
    }
    const int64_t t = blockIdx.x;
    if (PAIRS && t >= a.plan.tile_count[1]) return;
    if (!ROUTE && tid < a.top_k) to[tid] = PAIRS ? int(t) : a.plan.pair_row[t * a.top_k + tid];
    struct alignas(16) Group {
        T e[16];
    };
    const Group *row = reinterpret_cast<const Group *>(x + t * a.k);
    float top = 0.f, sum = 0.f, peak = 0.f;
    bool odd = false;  // an infinity or a NaN
    for (int g0 = 0; g0 < a.k / 16; g0 += kStageThreads) {
        float mine = 0.f;
        if (g0 + tid < a.k / 16) {
            const Group v = row[g0 + tid];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float f = fabsf(to_f32(v.e[i]));
                top = fmaxf(top, f);
                mine += f;
                odd |= !(f < INFINITY);
            }
        }
        if (F8) continue;
        sum += mine;
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);  // (a block of 128: eight groups)
        peak = fmaxf(peak, mine);
    }
    top = odd ? INFINITY : top;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
        peak = fmaxf(peak, __shfl_xor_sync(0xffffffffu, peak, o));
    }
    if (lane == 0) {
        part[0][warp] = top;
        part[1][warp] = sum;
        part[2][warp] = peak;
    }
    __syncthreads();
    sum = 0.f;
#pragma unroll
    for (int w = 0; w < kStageThreads / 32; ++w) {
        top = fmaxf(top, part[0][w]);
        sum += part[1][w];
        peak = fmaxf(peak, part[2][w]);
    }
    const int up = top < INFINITY ? min((F8 ? 7 : 14) - moe_log2(top), 126) : 0;
    const float by = moe_power(up);
    if (tid < a.top_k && to[tid] >= 0) {
        a.scale[to[tid]] = F8 && !(top < INFINITY) ? __uint_as_float(0x7fc00000u) : moe_power(-up);
        if (!F8) {  // (more by what sums of these and of the scales may have been rounded down, 2^-24 an addition)
            a.sum[to[tid]] = sum * (1.f + 0x1p-10f);
            a.peak[to[tid]] = peak * (1.f + 0x1p-10f);
        }
    }
    for (int g = tid; g < a.k / 16; g += kStageThreads) {
        const Group v = row[g];
        if constexpr (F8) {
            alignas(16) __nv_fp8_storage_t term[3][16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float rest = to_f32(v.e[i]) * by;
#pragma unroll
                for (int j = 0; j < 3; ++j) {
                    const __nv_fp8_storage_t b = __nv_cvt_float_to_fp8(rest, __NV_SATFINITE, __NV_E4M3);
                    term[j][moe_place8(i)] = b;
                    rest = (rest - __half2float(__half(__nv_cvt_fp8_to_halfraw(b, __NV_E4M3)))) * 16.f;
                }
            }
            for (int j = 0; j < a.top_k; ++j) {
                if (to[j] < 0) continue;
                uint8_t *dst = static_cast<uint8_t *>(a.staged) + int64_t(to[j]) * 3 * a.k + 16 * g;
#pragma unroll
                for (int i = 0; i < 3; ++i) *reinterpret_cast<uint4 *>(dst + int64_t(i) * a.k) = *reinterpret_cast<const uint4 *>(term[i]);
            }
        } else {
            __half2 hi[8], lo[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float p = to_f32(v.e[i]) * by, q = to_f32(v.e[i + 8]) * by;
                hi[i] = __floats2half2_rn(p, q);
                const float2 h = __half22float2(hi[i]);
                lo[i] = __floats2half2_rn((p - h.x) * kLowScale, (q - h.y) * kLowScale);
            }
            for (int j = 0; j < a.top_k; ++j) {
                if (to[j] < 0) continue;
                uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__half *>(a.staged) + int64_t(to[j]) * a.terms * a.k + 16 * g);
                dst[0] = reinterpret_cast<const uint4 *>(hi)[0];
                dst[1] = reinterpret_cast<const uint4 *>(hi)[1];
                if (a.terms == 2) {
                    dst += a.k / 8;
                    dst[0] = reinterpret_cast<const uint4 *>(lo)[0];
                    dst[1] = reinterpret_cast<const uint4 *>(lo)[1];
                }
            }
        }
    }
}

constexpr int kSumThreads = 256;

// out[t] = residual[t] + sum_j weight[t, j] y[row of (t, j)], four elements a thread.
template <typename T>
__global__ void __launch_bounds__(kSumThreads) moe_sum_kernel(MoeArgs a, MoePlan plan, const float *__restrict__ y) {
    const int64_t i = (int64_t(blockIdx.x) * kSumThreads + threadIdx.x) * 4;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (i >= a.tokens * a.width) return;
    const int64_t t = i / a.width, c = i - t * a.width;
    struct alignas(4 * sizeof(T)) Four {
        T e[4];
    };
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    if (a.residual) {
        const Four r = *reinterpret_cast<const Four *>(static_cast<const T *>(a.residual) + i);
#pragma unroll
        for (int j = 0; j < 4; ++j) s[j] = to_f32(r.e[j]);
    }
    constexpr int U = 8;  // pairs whose loads are in flight together
    for (int j0 = 0; j0 < a.top_k; j0 += U) {
        int row[U];
        float w[U];
        float4 v[U];
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int64_t p = t * a.top_k + min(j0 + j, a.top_k - 1);
            row[j] = j0 + j < a.top_k ? plan.pair_row[p] : -1;
            w[j] = a.weight[p];
        }
#pragma unroll
        for (int j = 0; j < U; ++j)
            if (row[j] >= 0) v[j] = *reinterpret_cast<const float4 *>(y + int64_t(row[j]) * a.width + c);
#pragma unroll
        for (int j = 0; j < U; ++j)
            if (row[j] >= 0) {
                s[0] = fmaf(w[j], v[j].x, s[0]);
                s[1] = fmaf(w[j], v[j].y, s[1]);
                s[2] = fmaf(w[j], v[j].z, s[2]);
                s[3] = fmaf(w[j], v[j].w, s[3]);
            }
    }
    Four o;
#pragma unroll
    for (int j = 0; j < 4; ++j) o.e[j] = from_f32<T>(s[j]);
    *reinterpret_cast<Four *>(static_cast<T *>(a.out) + i) = o;
}

size_t pad(size_t n) { return (n + 255) & ~size_t(255); }

// How a call of some size is computed: terms of an activation, columns of a tile.
//  * 16-bit activations of at most 16 rows an expert in the mean: three e4m3 terms (see moe.cuh).
//  * Else one binary16 term, or two of f32 activations, and columns by the staged rows that experts have in the mean: with
//    more columns codes are decoded less often, with fewer there is room for more decoded weights and more warps that decode.
// Measured (us a call in a graph; e4m3 / 32 / 64 / 96 columns of binary16; A: 8 of 128 experts of 2048 x 768, bf16,
// B: 2 of 8 of 4096 x 6144, f16, C: 2 of 16 of 1280 x 2816, f32):
//   rows    1 (16 tokens, 4)          4                       8                       12                      16
//   A   45 /  50 /  57 /  59    66 /  70 /  81 /  83    81 /  81 /  91 /  95    96 /  86 /  95 /  99   111 /  97 / 102 / 105
//   B   60 /  66 /  79 /  80    74 /  81 /  98 / 100    78 /  83 /  99 / 100    87 /  85 / 100 / 101   102 /  87 / 101 / 103
//   rows   24                         32                      48                      64                      96
//   A  140 / 111 / 111 / 115   172 / 131 / 124 / 125   231 / 165 / 147 / 147   292 / 204 / 173 / 169   420 / 282 / 229 / 219
//   B  147 /  97 / 105 / 107   171 / 116 / 108 / 110   223 / 154 / 122 / 120   277 / 171 / 146 / 132   378 / 238 / 197 / 173
//   C (two terms)  1: 26 / 29 / 29   8: 39 / 40 / 41   16: 47 / 47 / 46   24: 59 / 53 / 54   32: 67 / 58 / 60   64: 104 / 83 / 80
// Three terms pay up to 8 rows and cost 10 to 17 % at 12 to 16, where experts of more than 16 have a second tile; the border
// stands at 16, up to which a token's result is then the same whatever the tokens beside it.
struct Form {
    int terms, cols;
};
Form form_of(int dtype, int64_t pairs, int64_t experts) {
    const int64_t active = std::min(pairs, experts);
    if (dtype != TQ2_F32 && pairs <= 16 * active) return {3, 48};
    const int terms = dtype == TQ2_F32 ? 2 : 1;
    const int64_t rows = pairs * terms;
    return {terms, rows <= 16 * active ? 32 : rows <= 64 * active ? 64 : 96};
}

struct Workspace {
    MoePlan plan;
    uint8_t *staged_x, *staged_h;
    float *scale_x, *scale_h, *sum_x, *peak_x, *h, *y;
    int max_tiles, bound_rows, bound_blocks;  // features that a block bounds, blocks of an expert
    size_t bytes;

    // (Sizes are the largest that any form of this many pairs, or of fewer, takes.)
    Workspace(char *base, int64_t pairs, int64_t experts, int64_t width, int64_t ffn, int dtype) {
        size_t at = 0;
        auto take = [&](auto *&p, size_t n) {
            p = reinterpret_cast<std::remove_reference_t<decltype(p)>>(base + at);
            at += pad(n * sizeof(*p));
        };
        const Form form = form_of(dtype, pairs, experts);
        max_tiles = int(std::min(pairs, experts) + pairs / (form.cols / form.terms));  // each expert leaves less than one unfilled
        const int64_t few = dtype == TQ2_F32 ? 0 : std::min(pairs, 16 * experts);  // pairs of the three-term form, at most
        take(plan.tile_count, 2);
        take(plan.tiles, size_t(std::min(pairs, experts) + pairs / 16));
        take(plan.pair_row, size_t(pairs));
        take(plan.expert_rows, size_t(experts));
        bound_rows = std::max(8, int(kBoundScales / (width / kBlockW)) & ~7);
        bound_blocks = int((ffn + bound_rows - 1) / bound_rows);
        take(plan.bound, size_t(experts * bound_blocks));
        take(scale_x, size_t(pairs));
        take(scale_h, size_t(pairs));
        take(sum_x, size_t(pairs));
        take(peak_x, size_t(pairs));
        take(staged_x, size_t(std::max(pairs * (dtype == TQ2_F32 ? 4 : 2), few * 3) * width));
        take(staged_h, size_t(std::max(pairs * (dtype == TQ2_F32 ? 4 : 2), few * 3) * ffn));
        take(h, size_t(few * ffn));
        take(y, size_t(pairs * width));
        bytes = at;
    }
};

cudaError_t launch_plan(const MoeArgs &a, const Workspace &w, int64_t pairs, const Form &form, const LaunchCtx &ctx) {
    int cluster = 1;
    while (cluster < kPlanMaxCluster && pairs > cluster * kPlanPairs) cluster *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(cluster));
    cfg.blockDim = dim3(kPlanThreads);
    cfg.stream = ctx.stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = unsigned(cluster);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, moe_plan_kernel, a.expert, w.plan, int(pairs), a.experts, form.cols / form.terms, cluster,
                              ctx.status);
}

template <typename T>
cudaError_t launch(const MoeArgs &a, int dtype, void *ws, const LaunchCtx &ctx) {
    const int64_t pairs = a.tokens * a.top_k;
    const Form form = form_of(dtype, pairs, a.experts);
    const bool f8 = form.terms == 3;
    const Workspace w(static_cast<char *>(ws), pairs, a.experts, a.width, a.ffn, dtype);
    const SoaView gate_up = soa_view(a.gate_up, int64_t(a.experts) * 2 * a.ffn, a.width);
    const SoaView down = soa_view(a.down, int64_t(a.experts) * a.width, a.ffn);
    const bool route = pairs <= kFewPairs;  // sorted by the blocks that stage them
    cudaError_t e = route ? cudaSuccess : launch_plan(a, w, pairs, form, ctx);
    if (e != cudaSuccess) return e;
    StageArgs s = {};
    s.expert = a.expert;
    s.tile_rows = form.cols / form.terms;
    s.status = ctx.status;
    s.plan = w.plan;
    s.staged = w.staged_x;
    s.scale = w.scale_x;
    s.sum = w.sum_x;
    s.peak = w.peak_x;
    s.d = gate_up.d;
    s.ffn = a.ffn;
    s.bound_blocks = f8 ? 0 : w.bound_blocks;
    s.bound_rows = w.bound_rows;
    s.bound_lanes = 1;
    while (s.bound_lanes < 16 && s.bound_lanes * 2 * w.bound_rows <= kStageThreads) s.bound_lanes *= 2;
    s.tokens = a.tokens;
    s.k = a.width;
    s.top_k = a.top_k;
    s.terms = form.terms;
    s.experts = a.experts;
    const T *x = static_cast<const T *>(a.x);
    const dim3 stage_grid(unsigned(a.tokens + route + int64_t(a.experts) * s.bound_blocks));
    auto stage = f8 ? route ? moe_stage_kernel<T, true, false, true> : moe_stage_kernel<T, true, false, false>
                    : route ? moe_stage_kernel<T, false, false, true> : moe_stage_kernel<T, false, false, false>;
    const int bound_bytes = f8 ? 0 : 2 * w.bound_rows * (a.width / kBlockW) * int(sizeof(__half));  // (16 KB at most)
    e = launch_dependent(stage, stage_grid, kStageThreads, bound_bytes, ctx.stream, x, s);
    if (e != cudaSuccess) return e;
    MoeGemm g = {};
    g.plan = w.plan;
    g.pairs = pairs;
    g.experts = a.experts;
    g.terms = form.terms;
    g.cols = form.cols;
    g.max_tiles = w.max_tiles;
    g.bound_blocks = w.bound_blocks;
    g.qs = gate_up.qs;
    g.d = gate_up.d;
    g.staged = w.staged_x;
    g.scale = w.scale_x;
    g.sum = w.sum_x;
    g.peak = w.peak_x;
    g.out = w.h;
    g.staged_out = reinterpret_cast<__half *>(w.staged_h);
    g.scale_out = w.scale_h;
    g.rows = 2 * a.ffn;
    g.k = a.width;
    if ((e = launch_moe_gemm(g, true, ctx)) != cudaSuccess) return e;
    if (f8) {  // (e4m3 terms need the rows' largest values, not bounds of them)
        s.staged = w.staged_h;
        s.scale = w.scale_h;
        s.tokens = pairs;
        s.k = a.ffn;
        s.top_k = 1;
        e = launch_dependent(moe_stage_kernel<float, true, true, false>, dim3(unsigned(pairs)), kStageThreads, 0, ctx.stream,
                             static_cast<const float *>(w.h), s);
        if (e != cudaSuccess) return e;
    }
    g.qs = down.qs;
    g.d = down.d;
    g.staged = w.staged_h;
    g.scale = w.scale_h;
    g.out = w.y;
    g.rows = a.width;
    g.k = a.ffn;
    if ((e = launch_moe_gemm(g, false, ctx)) != cudaSuccess) return e;
    const int64_t blocks = (a.tokens * a.width / 4 + kSumThreads - 1) / kSumThreads;
    return launch_dependent(moe_sum_kernel<T>, dim3(unsigned(blocks)), kSumThreads, 0, ctx.stream, a, w.plan,
                            static_cast<const float *>(w.y));
}

}  // namespace

size_t moe_ws_bytes(int64_t tokens, int64_t top_k, int64_t experts, int64_t width, int64_t ffn, int dtype) {
    return Workspace(nullptr, tokens * top_k, experts, width, ffn, dtype).bytes;
}

cudaError_t launch_moe(const MoeArgs &a, int dtype, void *ws, const LaunchCtx &ctx) {
    switch (dtype) {
        case TQ2_F32: return launch<float>(a, dtype, ws, ctx);
        case TQ2_F16: return launch<__half>(a, dtype, ws, ctx);
        default: return launch<__nv_bfloat16>(a, dtype, ws, ctx);
    }
}

}  // namespace tq2
