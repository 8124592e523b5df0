// Mixture of ternary experts:
//     out[t] = residual[t] + sum_j weight[t, j] Down_e (silu(Gate_e x_t) * (Up_e x_t)),  e = expert[t, j].
//
// The (token, expert) pairs are sorted by expert (moe_plan_kernel), so that an expert's codes are read once for all its
// tokens; each pair's activations are staged as binary16 for the tensor cores (moe_stage_kernel), both products run as
// grouped products on them (moe_gemm.cu), and each token's pairs are summed in their order (moe_sum_kernel): no atomics,
// the same bits on every call.
#include <cstdint>

#include "dtype.cuh"
#include "moe.cuh"
#include "paged_attention.cuh"

namespace tq2 {
namespace {

constexpr int kPlanThreads = 1024, kPlanWarps = 32, kPlanAhead = 8;

// Exclusive sum over the block's threads of v; total: the sum.
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
        int x = part[lane];
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

// The pairs sorted by expert (in their order within one), and the tiles.  One block: warp w counts and places the pairs of
// the w-th part, 32 at a time.
__global__ void __launch_bounds__(kPlanThreads)
moe_plan_kernel(const int32_t *__restrict__ expert, MoePlan plan, int pairs, int experts, int tile_rows, unsigned int *status) {
    extern __shared__ int cnt[];  // [kPlanWarps][experts]
    __shared__ int part[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int i = threadIdx.x; i < kPlanWarps * experts; i += kPlanThreads) cnt[i] = 0;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __syncthreads();
    const int per = ((pairs + kPlanWarps - 1) / kPlanWarps + 31) / 32 * 32;
    const int first = min(pairs, warp * per), last = min(pairs, first + per);
    int *mine = cnt + warp * experts;
    bool bad = false;
    // 8 x 32 of them in flight, and kept where they are all there are
    int id[kPlanAhead];
    auto load = [&](int p0) {
#pragma unroll
        for (int i = 0; i < kPlanAhead; ++i) {
            const int p = p0 + 32 * i + lane;
            id[i] = p < last ? expert[p] : -1;
            if (id[i] < 0 || id[i] >= experts) {
                bad |= id[i] != -1;
                id[i] = -1;
            }
        }
    };
    for (int p0 = first; p0 < last; p0 += 32 * kPlanAhead) {
        load(p0);
#pragma unroll
        for (int i = 0; i < kPlanAhead; ++i) {
            if (p0 + 32 * i >= last) break;
            const uint32_t same = __match_any_sync(0xffffffffu, id[i]);
            if (id[i] >= 0 && lane == __ffs(same) - 1) mine[id[i]] += __popc(same);
            __syncwarp();
        }
    }
    report_bad(bad, status);
    __syncthreads();
    const int e = threadIdx.x;
    int total = 0;
    if (e < experts)
        for (int w = 0; w < kPlanWarps; ++w) {
            const int c = cnt[w * experts + e];
            cnt[w * experts + e] = total;
            total += c;
        }
    int rows, tiles;
    const int at = block_scan(total, part, &rows);
    const int n_tiles = (total + tile_rows - 1) / tile_rows;
    const int tile0 = block_scan(n_tiles, part, &tiles);
    if (e < experts)
        for (int w = 0; w < kPlanWarps; ++w) cnt[w * experts + e] += at;
    for (int i = 0; i < n_tiles; ++i)
        plan.tiles[tile0 + i] = MoeTile{e, at + i * tile_rows, min(tile_rows, total - i * tile_rows), 0};
    if (threadIdx.x == 0) {
        plan.counts[0] = tiles;
        plan.counts[1] = rows;
    }
    __syncthreads();
    for (int p0 = first; p0 < last; p0 += 32 * kPlanAhead) {
        if (last - first > 32 * kPlanAhead) load(p0);
#pragma unroll
        for (int i = 0; i < kPlanAhead; ++i) {
            if (p0 + 32 * i >= last) break;
            const int p = p0 + 32 * i + lane, x = id[i];
            const uint32_t same = __match_any_sync(0xffffffffu, x);
            int row = -1;
            if (x >= 0) {
                row = mine[x] + __popc(same & ((1u << lane) - 1));
                plan.row_pair[row] = p;
            }
            __syncwarp();
            if (x >= 0 && lane == __ffs(same) - 1) mine[x] += __popc(same);
            __syncwarp();
            if (p < last) plan.pair_row[p] = row;
        }
    }
}

constexpr int kStageThreads = 128;

// Stages a row a block: binary16 terms of the row times the power of two that brings its largest value between 2^14 and
// 2^15 (no value overflows, and one 2^-28 of the largest still has all its bits), in the products' order; scale is the
// power that undoes it.  GATHER: row r is that of the token of pair row_pair[r]; else row r of the input.
template <typename T, bool GATHER>
__global__ void __launch_bounds__(kStageThreads)
moe_stage_kernel(const T *__restrict__ in, MoePlan plan, __half *__restrict__ staged, float *__restrict__ scale, int k,
                 int top_k, int terms) {
    __shared__ float part[kStageThreads / 32];
    const int r = blockIdx.x;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (r >= plan.counts[1]) return;
    const T *row = in + int64_t(GATHER ? plan.row_pair[r] / top_k : r) * k;
    auto load = [&](int g, float (&v)[16]) {
        struct alignas(16) Group {
            T e[16];
        };
        const Group x = reinterpret_cast<const Group *>(row)[g];
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = to_f32(x.e[i]);
    };
    float top = 0.f;
    bool odd = false;  // an infinity or a NaN
    for (int g = threadIdx.x; g < k / 16; g += kStageThreads) {
        float v[16];
        load(g, v);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            top = fmaxf(top, fabsf(v[i]));
            odd |= !(fabsf(v[i]) < INFINITY);
        }
    }
    top = odd ? INFINITY : top;
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kStageThreads / 32; ++w) top = fmaxf(top, part[w]);
    // largest value 2^(e - 127) * [1, 2): times 2^(14 - (e - 127)), exponents kept to what f32 holds
    const int e = int(__float_as_uint(top) >> 23);
    const int up = top < INFINITY ? min(14 - (e - 127), 126) : 0;
    const float by = __uint_as_float(uint32_t(up + 127) << 23);
    if (threadIdx.x == 0) scale[r] = __uint_as_float(uint32_t(max(127 - up, 1)) << 23);
    for (int g = threadIdx.x; g < k / 16; g += kStageThreads) {
        float v[16];
        load(g, v);
        __half2 hi[8], lo[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float a = v[i] * by, b = v[i + 8] * by;
            hi[i] = __floats2half2_rn(a, b);
            const float2 h = __half22float2(hi[i]);
            lo[i] = __floats2half2_rn(a - h.x, b - h.y);
        }
        uint4 *to = reinterpret_cast<uint4 *>(staged + int64_t(r) * terms * k + 16 * g);
        to[0] = reinterpret_cast<const uint4 *>(hi)[0];
        to[1] = reinterpret_cast<const uint4 *>(hi)[1];
        if (terms == 2) {
            to = reinterpret_cast<uint4 *>(staged + (int64_t(r) * terms + 1) * k + 16 * g);
            to[0] = reinterpret_cast<const uint4 *>(lo)[0];
            to[1] = reinterpret_cast<const uint4 *>(lo)[1];
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
    for (int j = 0; j < a.top_k; ++j) {
        const int64_t p = t * a.top_k + j;
        const int row = plan.pair_row[p];
        if (row < 0) continue;
        const float w = a.weight[p];
        const float4 v = *reinterpret_cast<const float4 *>(y + int64_t(row) * a.width + c);
        s[0] = fmaf(w, v.x, s[0]);
        s[1] = fmaf(w, v.y, s[1]);
        s[2] = fmaf(w, v.z, s[2]);
        s[3] = fmaf(w, v.w, s[3]);
    }
    Four o;
#pragma unroll
    for (int j = 0; j < 4; ++j) o.e[j] = from_f32<T>(s[j]);
    *reinterpret_cast<Four *>(static_cast<T *>(a.out) + i) = o;
}

size_t pad(size_t n) { return (n + 255) & ~size_t(255); }

// Columns of a tile.  With 128 a tile's codes are decoded for twice the tokens; with 64 more warps decode, which is what
// counts where experts have few.
int tile_cols(int64_t pairs, int64_t experts, int terms) { return pairs * terms > 64 * std::min(pairs, experts) ? 128 : 64; }

struct Workspace {
    MoePlan plan;
    __half *staged_x, *staged_h;
    float *scale_x, *scale_h, *h, *y;
    int max_tiles, cols;
    size_t bytes;

    Workspace(char *base, int64_t pairs, int64_t experts, int64_t width, int64_t ffn, int terms) {
        size_t at = 0;
        auto take = [&](auto *&p, size_t n) {
            p = reinterpret_cast<std::remove_reference_t<decltype(p)>>(base + at);
            at += pad(n * sizeof(*p));
        };
        cols = tile_cols(pairs, experts, terms);
        const int64_t tile_rows = cols / terms;
        max_tiles = int(std::min(pairs, experts) + pairs / tile_rows);  // each expert leaves less than one unfilled
        take(plan.counts, 2);
        take(plan.tiles, size_t(max_tiles));
        take(plan.row_pair, size_t(pairs));
        take(plan.pair_row, size_t(pairs));
        take(scale_x, size_t(pairs));
        take(scale_h, size_t(pairs));
        take(staged_x, size_t(pairs * terms * width));
        take(h, size_t(pairs * ffn));
        take(staged_h, size_t(pairs * terms * ffn));
        take(y, size_t(pairs * width));
        bytes = at;
    }
};

int terms_of(int dtype) { return dtype == TQ2_F32 ? 2 : 1; }

template <typename T>
cudaError_t launch(const MoeArgs &a, int dtype, void *ws, const LaunchCtx &ctx) {
    const int64_t pairs = a.tokens * a.top_k;
    const int terms = terms_of(dtype);
    const Workspace w(static_cast<char *>(ws), pairs, a.experts, a.width, a.ffn, terms);
    const size_t plan_smem = size_t(kPlanWarps) * size_t(a.experts) * 4;
    cudaError_t e = cudaFuncSetAttribute(moe_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(plan_smem));
    if (e == cudaSuccess)
        e = launch_dependent(moe_plan_kernel, dim3(1), kPlanThreads, int(plan_smem), ctx.stream, a.expert, w.plan, int(pairs),
                             a.experts, w.cols / terms, ctx.status);
    if (e == cudaSuccess)
        e = launch_dependent(moe_stage_kernel<T, true>, dim3(unsigned(pairs)), kStageThreads, 0, ctx.stream,
                             static_cast<const T *>(a.x), w.plan, w.staged_x, w.scale_x, a.width, a.top_k, terms);
    if (e != cudaSuccess) return e;
    MoeGemm g = {};
    g.plan = w.plan;
    g.pairs = pairs;
    g.experts = a.experts;
    g.terms = terms;
    g.cols = w.cols;
    g.max_tiles = w.max_tiles;
    SoaView v = soa_view(a.gate_up, int64_t(a.experts) * 2 * a.ffn, a.width);
    g.qs = v.qs;
    g.d = v.d;
    g.staged = w.staged_x;
    g.scale = w.scale_x;
    g.out = w.h;
    g.rows = 2 * a.ffn;
    g.k = a.width;
    if ((e = launch_moe_gemm(g, true, ctx)) != cudaSuccess) return e;
    e = launch_dependent(moe_stage_kernel<float, false>, dim3(unsigned(pairs)), kStageThreads, 0, ctx.stream,
                         static_cast<const float *>(w.h), w.plan, w.staged_h, w.scale_h, a.ffn, 1, terms);
    if (e != cudaSuccess) return e;
    v = soa_view(a.down, int64_t(a.experts) * a.width, a.ffn);
    g.qs = v.qs;
    g.d = v.d;
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
    return Workspace(nullptr, tokens * top_k, experts, width, ffn, terms_of(dtype)).bytes;
}

cudaError_t launch_moe(const MoeArgs &a, int dtype, void *ws, const LaunchCtx &ctx) {
    switch (dtype) {
        case TQ2_F32: return launch<float>(a, dtype, ws, ctx);
        case TQ2_F16: return launch<__half>(a, dtype, ws, ctx);
        default: return launch<__nv_bfloat16>(a, dtype, ws, ctx);
    }
}

}  // namespace tq2
