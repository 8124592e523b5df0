// Grouped ternary product of a mixture of experts on the tcgen05 tensor cores:
//     out[row, f] = sum_k x[row, k] W_e[f, k]   for the rows of each expert e, or silu(gate) * up of two such.
//
// Computed transposed, W x^T: an item is 128 weight rows of one expert (the MMA's M) times a tile of up to 128 staged
// rows of its tokens (N, any multiple of 16), so that the codes of an expert are read once for a tile of tokens however
// few they are.
//
//  * The weights never touch shared memory decoded.  A thread takes one weight row, masks pairs of codes c out of its
//    words into binary16 numbers 2^n + c (one AND-OR a pair), subtracts 2^n + 1 (one packed subtraction, exact) and stores
//    the results to tensor memory, which the MMA reads as its A operand.  (Left as they are masked out, as subnormal
//    numbers, they would save nothing: the tensor core aligns products by the operands' exponents, and f32 sums lost ten
//    bits.)
//  * The block scale d stays out of the operands: each 128-weight block is a product of its own (eight MMAs) into one of
//    two accumulators, and d times it is added to the running sums in registers (f32).  So operands are exact, and what
//    is rounded is the activations' staging and the sums.
//  * Copies: codes by TMA, 512 weights of 128 rows a stage (64 KB in flight an SM); activations by TMA, 128 features of a
//    tile's rows a stage.
//  * Roles: warp 0 codes, warp 1 MMAs (owns tensor memory), warp 2 activations, warps 4-7 decode, warps 8-15 scale and
//    sum (columns 0-63 and 64-127).  One persistent CTA an SM.  Every wait is bounded; a timeout sets the status word and the
//    CTA drains its copies and MMAs before it leaves.
#include <cstdint>

#include "moe.cuh"
#include "paged_attention.cuh"

namespace tq2 {
namespace {

constexpr int kThreads = 512;
constexpr int W_CODES = 0, W_MMA = 1, W_ACT = 2, W_DECODE = 4, W_SUM = 8;
constexpr int kCodeStages = 4, kCodeK = 512, kCodeBytes = 128 * kCodeK / 4;  // 16 KB
constexpr int kActStages = 4, kActBytes = kMoeCols * kBlockW * 2;             // 32 KB: two halves of 64 features
constexpr int kABufs = 4, kACols = kBlockW / 2, kDBufs = 2;
constexpr uint32_t kTmemCols = 512, kACol = kDBufs * kMoeCols;
static_assert(kACol + kABufs * kACols <= kTmemCols, "TMEM budget");

struct Ctl {
    uint64_t c_full[kCodeStages], c_empty[kCodeStages];
    uint64_t x_full[kActStages], x_empty[kActStages];
    uint64_t a_full[kABufs], a_empty[kABufs];
    uint64_t d_full[kDBufs], d_empty[kDBufs];
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
};
constexpr int kOffAct = kCodeStages * kCodeBytes, kOffCtl = kOffAct + kActStages * kActBytes;
constexpr int kSmem = kOffCtl + int(sizeof(Ctl)) + 1024;
static_assert(kSmem <= 232448, "shared memory budget");

__device__ __forceinline__ uint64_t desc_k(uint32_t saddr) {  // K-major, 128-byte swizzle: rows 128 B, 8-row groups 1024 B
    return uint64_t((saddr & 0x3FFFFu) >> 4) | (uint64_t(1) << 16) | (uint64_t(1024 >> 4) << 32) | (uint64_t(1) << 46) |
           (uint64_t(2) << 61);
}

__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap *map, int x, int y, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_u32(bar))
        : "memory");
}

// D[tmem] (+)= A[tmem] * B[smem], A's lane = row, column c = elements 2c, 2c + 1
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void tm_ld32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tm_st32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tm_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Four words of 16 codes as 32 pairs of binary16 numbers code - 1: pair i of a word is its codes i and i + 8.  They stand at
// bits 2 i of each half; i < 5 within a binary16's mantissa, the others after a shift by 10.
__device__ __forceinline__ void decode(const uint4 &w, uint32_t (&r)[32]) {
    const uint32_t word[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t high = word[j] >> 10;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int e = i < 5 ? i : i - 5;
            const uint32_t exponent = uint32_t(25 - 2 * e) << 10;  // of 2^(10 - 2 e): a code at bit 2 e counts ones
            const uint32_t v = ((i < 5 ? word[j] : high) & (0x00030003u << (2 * e))) | exponent | exponent << 16;
            const __half2 s = __hsub2(*reinterpret_cast<const __half2 *>(&v), __float2half2_rn(float((1 << (10 - 2 * e)) + 1)));
            r[8 * j + i] = *reinterpret_cast<const uint32_t *>(&s);
        }
    }
}

// An item's place: its tile and its 128 weight rows.
struct Item {
    MoeTile tile;
    int part;     // which 128 rows
    int cols;     // MMA columns: staged rows, to a multiple of 16
};
__device__ __forceinline__ Item item_of(const MoeGemm &g, int i, int parts) {
    Item it;
    const int4 t = *reinterpret_cast<const int4 *>(g.plan.tiles + i / parts);
    it.tile = MoeTile{uniform(t.x), uniform(t.y), uniform(t.z), 0};
    it.part = uniform(i % parts);
    it.cols = (it.tile.n * g.terms + 15) & ~15;
    return it;
}

// x / (1 + exp(-x)), with the fast exponential and quotient (relative error about 2^-21)
__device__ __forceinline__ float silu(float x) { return __fdividef(x, 1.f + __expf(-x)); }

template <bool GATE_UP>
__global__ void __launch_bounds__(kThreads, 1)
moe_gemm_kernel(const __grid_constant__ CUtensorMap cmap, const __grid_constant__ CUtensorMap xmap, const MoeGemm g,
                unsigned int *status, uint64_t wait_ns) {
    extern __shared__ __align__(1024) uint8_t raw[];
    uint8_t *smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    Ctl *ctl = reinterpret_cast<Ctl *>(smem + kOffCtl);
    const int warp = uniform(int(threadIdx.x >> 5)), lane = threadIdx.x & 31;
    volatile int *abort_flag = &ctl->abort;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kCodeStages; ++s) {
            mbar_init(&ctl->c_full[s], 1);
            mbar_init(&ctl->c_empty[s], 4);
        }
        for (int s = 0; s < kActStages; ++s) {
            mbar_init(&ctl->x_full[s], 1);
            mbar_init(&ctl->x_empty[s], 1);
        }
        for (int s = 0; s < kABufs; ++s) {
            mbar_init(&ctl->a_full[s], 4);
            mbar_init(&ctl->a_empty[s], 1);
        }
        for (int s = 0; s < kDBufs; ++s) {
            mbar_init(&ctl->d_full[s], 1);
            mbar_init(&ctl->d_empty[s], 8);
        }
        mbar_init(&ctl->drain, 1);
        ctl->abort = 0;
        fence_mbarrier_init();
        fence_proxy_async_smem();
    }
    if (warp == W_MMA) {
        tmem_alloc(&ctl->tmem_base, kTmemCols);
        tmem_relinquish();
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = uint32_t(uniform(int(ctl->tmem_base)));
    const int parts = g.rows / 128, nb = uniform(g.k / kBlockW);
    const int items = uniform(g.plan.counts[0] * parts);
    auto wait_on = [&](uint64_t *bar, uint32_t parity) {
        return bool(__all_sync(0xffffffffu, wait_phase(bar, parity, abort_flag, wait_ns, status)));
    };

    if (warp == W_CODES) {
        int n = 0;  // stages filled
        bool ok = true;
        for (int i = blockIdx.x; ok && i < items; i += gridDim.x) {
            const Item it = item_of(g, i, parts);
            const int row = it.tile.expert * g.rows;
            const int y0 = row + (GATE_UP ? 64 : 128) * it.part, y1 = GATE_UP ? y0 + g.rows / 2 : y0 + 64;
            for (int k = 0; k < g.k; k += kCodeK, ++n) {
                const int s = n % kCodeStages;
                if (n >= kCodeStages && !(ok = wait_on(&ctl->c_empty[s], (n / kCodeStages - 1) & 1))) break;
                if (elect_one()) {
                    mbar_expect_tx(&ctl->c_full[s], kCodeBytes);
                    const uint32_t dst = smem_u32(smem) + uint32_t(s * kCodeBytes);
                    tma_2d(dst, &cmap, k / 4, y0, &ctl->c_full[s]);
                    tma_2d(dst + kCodeBytes / 2, &cmap, k / 4, y1, &ctl->c_full[s]);
                }
                __syncwarp();
            }
        }
        if (lane == 0)  // every copy lands before the CTA ends
            for (int j = max(0, n - kCodeStages); j < n; ++j)
                mbar_wait_bounded(&ctl->c_full[j % kCodeStages], (j / kCodeStages) & 1, drain_ns(wait_ns), status);
        __syncwarp();
    } else if (warp == W_ACT) {
        int n = 0;
        bool ok = true;
        for (int i = blockIdx.x; ok && i < items; i += gridDim.x) {
            const Item it = item_of(g, i, parts);
            for (int b = 0; b < nb; ++b, ++n) {
                const int s = n % kActStages;
                if (n >= kActStages && !(ok = wait_on(&ctl->x_empty[s], (n / kActStages - 1) & 1))) break;
                if (elect_one()) {
                    mbar_expect_tx(&ctl->x_full[s], uint32_t(it.cols) * 256);
                    const uint32_t dst = smem_u32(smem) + uint32_t(kOffAct + s * kActBytes);
                    for (int c = 0; c < it.cols; c += 16)
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            tma_2d(dst + uint32_t(h * (kActBytes / 2) + c * 128), &xmap, b * kBlockW + 64 * h,
                                   it.tile.row0 * g.terms + c, &ctl->x_full[s]);
                }
                __syncwarp();
            }
        }
        if (lane == 0)
            for (int j = max(0, n - kActStages); j < n; ++j)
                mbar_wait_bounded(&ctl->x_full[j % kActStages], (j / kActStages) & 1, drain_ns(wait_ns), status);
        __syncwarp();
    } else if (warp == W_MMA) {
        int n = 0;  // blocks
        bool ok = true;
        for (int i = blockIdx.x; ok && i < items; i += gridDim.x) {
            const Item it = item_of(g, i, parts);
            const uint32_t idesc = uint32_t(uniform(int((1u << 4) | (uint32_t(it.cols >> 3) << 17) | (uint32_t(128 >> 4) << 24))));
            for (int b = 0; b < nb; ++b, ++n) {
                const int sx = n % kActStages, sa = n % kABufs, sd = n % kDBufs;
                if (n >= kDBufs) ok = wait_on(&ctl->d_empty[sd], (n / kDBufs - 1) & 1);
                ok = ok && wait_on(&ctl->x_full[sx], (n / kActStages) & 1) && wait_on(&ctl->a_full[sa], (n / kABufs) & 1);
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t db = desc_k(smem_u32(smem) + uint32_t(kOffAct + sx * kActBytes));
                    const uint32_t d = tmem + uint32_t(sd * kMoeCols), at = tmem + kACol + uint32_t(sa * kACols);
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        mma_ts(d, at + uint32_t(kk * 8), db + uint64_t((kk >> 2) * (kActBytes / 2 >> 4) + 2 * (kk & 3)), idesc, kk > 0);
                    tc_commit(&ctl->a_empty[sa]);
                    tc_commit(&ctl->x_empty[sx]);
                    tc_commit(&ctl->d_full[sd]);
                }
                __syncwarp();
            }
        }
        if (elect_one()) tc_commit(&ctl->drain);
        __syncwarp();
    } else if (warp >= W_DECODE && warp < W_SUM) {
        const int q = warp & 3;
        // the row of this thread's lane among the stage's 128: gate rows in lanes 0-15, the up rows of the same features above
        const int r = GATE_UP ? (lane < 16 ? 16 * q + lane : 48 + 16 * q + lane) : 32 * q + lane;
        int n = 0, stage = 0;
        bool ok = true;
        for (int i = blockIdx.x; ok && i < items; i += gridDim.x) {
            for (int b = 0; b < nb; ++b, ++n) {
                const int sc = stage % kCodeStages, sa = n % kABufs;
                if ((b & 3) == 0 && !(ok = wait_on(&ctl->c_full[sc], (stage / kCodeStages) & 1))) break;
                const uint8_t *row = smem + sc * kCodeBytes + r * 128;
                uint4 w[2];
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    w[j] = *reinterpret_cast<const uint4 *>(row + (((2 * (b & 3) + j) ^ (r & 7)) << 4));
                if ((b & 3) == 3 || b == nb - 1) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ctl->c_empty[sc]);
                    ++stage;
                }
                if (n >= kABufs && !(ok = wait_on(&ctl->a_empty[sa], (n / kABufs - 1) & 1))) break;
                tc_fence_after();
                const uint32_t at = tmem + kACol + uint32_t(sa * kACols) + (uint32_t(q * 32) << 16);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    uint32_t v[32];
                    decode(w[j], v);
                    tm_st32(at + uint32_t(32 * j), v);
                }
                tm_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl->a_full[sa]);
            }
        }
    } else if (warp >= W_SUM) {
        const int q = warp & 3, col0 = 64 * ((warp - W_SUM) >> 2);
        int n = 0;
        bool ok = true;
        for (int i = blockIdx.x; ok && i < items; i += gridDim.x) {
            const Item it = item_of(g, i, parts);
            const int row = it.tile.expert * g.rows + (GATE_UP ? 64 * it.part + 16 * q + (lane & 15) + (lane < 16 ? 0 : g.rows / 2)
                                                              : 128 * it.part + 32 * q + lane);
            const __half *dp = g.d + int64_t(row) * nb;
            float acc[64];
#pragma unroll
            for (int c = 0; c < 64; ++c) acc[c] = 0.f;
            float dn = __half2float(dp[0]);
            for (int b = 0; b < nb; ++b, ++n) {
                const int sd = n % kDBufs;
                const float d = dn;
                if (b + 1 < nb) dn = __half2float(dp[b + 1]);
                if (!(ok = wait_on(&ctl->d_full[sd], (n / kDBufs) & 1))) break;
                tc_fence_after();
                const uint32_t at = tmem + uint32_t(sd * kMoeCols + col0) + (uint32_t(q * 32) << 16);
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    if (col0 + 32 * h < it.cols) {
                        uint32_t v[32];
                        tm_ld32(at + uint32_t(32 * h), v);
#pragma unroll
                        for (int c = 0; c < 32; ++c) acc[32 * h + c] = fmaf(d, __uint_as_float(v[c]), acc[32 * h + c]);
                    }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl->d_empty[sd]);
            }
            if (!ok) break;
            // rows of this warp's columns (the staged terms of one side by side)
            auto finish = [&](auto two) {
                constexpr int S = decltype(two)::value;
                const int r0 = col0 / S, left = it.tile.n - r0;
                const float *scale = g.scale + it.tile.row0 + r0;
                const int features = GATE_UP ? g.rows / 2 : g.rows;
                float *out = g.out + int64_t(it.tile.row0 + r0) * features;
                if (S == 2) {
#pragma unroll
                    for (int c = 0; c < 32; ++c) acc[c] = acc[2 * c] + acc[2 * c + 1];
                }
                if (GATE_UP) {
                    out += 64 * it.part + 16 * q + (lane & 15);
                    const bool up = lane >= 16;
#pragma unroll
                    for (int c = 0; c < 64 / S; c += 2) {
                        if (c >= left) break;
                        // lanes 0-15 finish row c, lanes 16-31 row c + 1
                        const float s = scale[min(c + up, left - 1)];
                        const float other = __shfl_xor_sync(0xffffffffu, up ? acc[c] : acc[c + 1], 16);
                        const float gate = (up ? other : acc[c]) * s, ups = (up ? acc[c + 1] : other) * s;
                        if (c + up < left) out[int64_t(c + up) * features] = silu(gate) * ups;
                    }
                } else {
                    out += 128 * it.part + 32 * q + lane;
#pragma unroll
                    for (int c = 0; c < 64 / S; ++c)
                        if (c < left) out[int64_t(c) * features] = acc[c] * scale[c];
                }
            };
            if (g.terms == 2)
                finish(std::integral_constant<int, 2>{});
            else
                finish(std::integral_constant<int, 1>{});
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == W_MMA) {
        // every issued MMA must be complete before TMEM is released
        if (lane == 0) mbar_wait_bounded(&ctl->drain, 0, drain_ns(wait_ns), status);
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

cudaError_t map_2d(CUtensorMap *map, CUtensorMapDataType type, const void *base, int64_t inner, int64_t rows, int64_t row_bytes,
                   int box_inner, int box_rows, CUtensorMapL2promotion promote) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return cudaErrorNotSupported;
    const cuuint64_t dims[2] = {cuuint64_t(inner), cuuint64_t(rows)}, strides[1] = {cuuint64_t(row_bytes)};
    const cuuint32_t box[2] = {cuuint32_t(box_inner), cuuint32_t(box_rows)}, step[2] = {1, 1};
    if (enc(map, type, 2, const_cast<void *>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, promote, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_moe_gemm(const MoeGemm &g, bool gate_up, const LaunchCtx &ctx) {
    CUtensorMap cmap, xmap;
    cudaError_t e = map_2d(&cmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, g.qs, g.k / 4, int64_t(g.experts) * g.rows, g.k / 4, 128, 64,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
    if (e == cudaSuccess)
        e = map_2d(&xmap, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, g.staged, g.k, g.pairs * g.terms, int64_t(g.k) * 2, 64, 16,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_128B);
    if (e != cudaSuccess) return e;
    auto kernel = gate_up ? moe_gemm_kernel<true> : moe_gemm_kernel<false>;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    const int64_t items = int64_t(g.max_tiles) * (g.rows / 128);
    const unsigned grid = unsigned(std::min<int64_t>(items, ctx.num_sms));
    return launch_dependent(kernel, dim3(grid), kThreads, kSmem, ctx.stream, cmap, xmap, g, ctx.status, ctx.wait_ns);
}

}  // namespace tq2
