// Attention of a step's new tokens over a paged key/value cache: many query rows
// per (sequence, key head), on the tcgen05 tensor cores.
//
// Mathematics: the online softmax of attention_paged.cu with the query rows in M.
// The rows of a sequence and key head are its new tokens times the query heads of
// the group, row = token * G + head, so a 128-row tile of a chunk reads each key
// for all G heads at once.
//
//  * A CTA owns up to 256 consecutive rows (two tiles) of one (sequence, key head)
//    and a chunk of keys, in blocks of 128.  Warps 0 and 12 copy K and V through
//    two-stage rings by paged tensor copies (boxes of rows inside one page); warps 1 and
//    2 issue the MMAs of lane 0 and 1 (below); warp 3 looks after V; warps 4-7 and 8-11
//    are the lanes' softmax groups, one thread per row (= tensor-memory lane).
//  * Lanes: with two tiles, lane w is tile w and walks every block; with one tile, lane
//    w walks the blocks 2i + w, so one tile keeps both softmax groups busy as well (they
//    meet at the end).  A lane walks in steps of 64 keys (half a block), each step with
//    its own half of the lane's score columns: the softmax of step u runs while the
//    MMAs of step u + 1 are queued, and neither waits for the other's round trip.  A
//    lane's MMAs, a step: P V of step u, then S of step u + 2 over the same columns
//    (MMAs of one thread execute in issue order).  Each lane has an issuing warp of its
//    own, so that the tensor core runs one lane's MMAs while the other's thread waits
//    (a wait takes 80 to 200 cycles even where its phase is complete).
//  * Tensor memory: S of lane w, step u at columns 128 w + 64 (u & 1), O of lane w at
//    256 + 128 w.  P overwrites S in the cache's type (32 columns); for an f32 output the
//    weights' remainder follows as a second term in the other 32.
//  * V stays as it lies in the cache, [key][feature]: the second MMA's B operand is
//    MN-major, with the feature halves 16 KB apart (leading offset) and 8-key groups 1 KB
//    apart (stride offset).  No transposed copy of V exists.
//  * V's slots that no row sees are zeroed in shared memory, and where only some rows
//    see a key, values that are not finite are zeroed there and added, at the end, to
//    the rows that see them (0 * NaN is NaN).
// Every wait is bounded; a timeout sets the device status word and the CTA drains
// and exits.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include <cuda_bf16.h>

#include "paged_attention.cuh"

namespace tq2 {
namespace {

constexpr int kRows = 128;      // rows of a tile (MMA M)
constexpr int kBlock = 128;     // keys of a block (copies)
constexpr int kStep = 64;       // keys of a step (MMAs, softmax)
constexpr int kCtaRows = 2 * kRows;
constexpr int kThreads = 416;
constexpr int kMaxSplits = 64;
constexpr int kMinBlocks = 4;   // blocks a chunk, at least
constexpr uint32_t kTmemCols = 512, kOCol = 256;
constexpr float kLazy = 8.f;    // log2 growth of the maximum that O is rescaled for
constexpr int W_K = 0, W_MMA = 1, W_SOFT = 4, W_V = 12;  // W_MMA + lane; warp 3 looks after V

template <int DP>
struct ChunkLayout {
    static constexpr int HALVES = DP / 64;
    static constexpr int HALF = 128 * 128;            // 128 rows x 64 features, swizzled
    static constexpr int TILE = HALF * HALVES;        // Q tile, K block, V block
    static constexpr int OFF_K = 2 * TILE, OFF_V = OFF_K + 2 * TILE;
    static constexpr int OFF_CTL = OFF_V + 2 * TILE;
    static constexpr int OFF_ML = OFF_CTL + 256;      // m, l of group 1 (one tile)
    static constexpr int BYTES = OFF_ML + 2 * kRows * 4 + 1024;
    static constexpr int MPAD = DP + 4;               // f32 row of the groups' exchange, over Q and K
    static_assert(kRows * MPAD * 4 <= OFF_V, "the exchange reuses Q and K");
    static_assert(BYTES <= 232448, "shared memory budget");
};

struct ChunkCtl {
    uint64_t q_ready, k_full[2], k_empty[2], v_full[2], v_ready[2], v_empty[2];
    uint64_t s_full[2][2], p_full[2][2], o_done[2], drain;  // [lane][step & 1]
    uint32_t tmem_base;
    int abort, poisoned;
};
static_assert(sizeof(ChunkCtl) <= 256, "control block");

// Matrix descriptors (128-byte swizzle).  K-major: rows 128 B apart, 8-row groups
// 1024 B.  MN-major: 64 features contiguous, keys 128 B apart; 8-key groups 1024 B
// (stride offset), the next 64 features `HALF` bytes on (leading offset).
__device__ __forceinline__ uint64_t desc_k(uint32_t saddr) {
    return uint64_t((saddr & 0x3FFFFu) >> 4) | (uint64_t(1) << 16) | (uint64_t(1024 >> 4) << 32) | (uint64_t(1) << 46) |
           (uint64_t(2) << 61);
}
__device__ __forceinline__ uint64_t desc_mn(uint32_t saddr, uint32_t half) {
    return uint64_t((saddr & 0x3FFFFu) >> 4) | (uint64_t(half >> 4) << 16) | (uint64_t(1024 >> 4) << 32) |
           (uint64_t(1) << 46) | (uint64_t(2) << 61);
}

// D[tmem] (+)= A[tmem] * B[smem], A read from tensor memory (lane = row, column c =
// elements 2c, 2c + 1)
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
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
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
// Waits for this thread's loads; ties the registers to the wait, so that nothing that
// uses them moves ahead of it.
__device__ __forceinline__ void tm_wait_ld(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                   "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]),
                   "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
                   "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
                 :
                 : "memory");
}
__device__ __forceinline__ void tm_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float max3(float a, float b, float c) {  // (a NaN operand is ignored)
    float y;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}
__device__ __forceinline__ uint64_t pair(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t r, float &a, float &b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// The sequence and first row of CTA slot `slot`: sequences and their row tiles from
// the last to the first (the last tiles of a causal prompt are the longest).  One
// warp; false if the slot is past the last tile.
__device__ __forceinline__ bool find_rows(const BatchView &bt, int G, int slot, int &b_out, int &row0, unsigned int *status) {
    const int lane = threadIdx.x & 31;
    for (int top = bt.seqs; top > 0; top -= 32) {
        const int b = top - 1 - lane;
        int tiles = 0;
        if (b >= 0) {
            bool bad = false;
            const SeqSpan sp = seq_span(bt, b, bad);
            report_bad(bad, status);
            tiles = int((int64_t(sp.n) * G + kCtaRows - 1) / kCtaRows);
        }
        int upto = tiles;  // inclusive sums over the lanes
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, upto, d);
            if (lane >= d) upto += x;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, slot < upto);
        if (hit) {
            const int l = __ffs(hit) - 1;
            b_out = top - 1 - l;
            row0 = (__shfl_sync(0xffffffffu, upto, l) - 1 - slot) * kCtaRows;
            return true;
        }
        slot -= __shfl_sync(0xffffffffu, upto, 31);
    }
    return false;
}

template <typename T, typename TO, int DP>
__global__ void __launch_bounds__(kThreads, 1)
paged_chunk_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, const PagedArgs a,
                   const KeyPlan plan, float *__restrict__ part_o, float2 *__restrict__ part_ml, unsigned int *status,
                   uint64_t wait_ns) {
    using L = ChunkLayout<DP>;
    constexpr bool SPLIT_P = sizeof(TO) == 4;
    extern __shared__ uint8_t chunk_raw[];
    const uint32_t raw = smem_u32(chunk_raw), pad = (1024u - (raw & 1023u)) & 1023u, base = raw + pad;
    uint8_t *smem = chunk_raw + pad;
    ChunkCtl *ctl = reinterpret_cast<ChunkCtl *>(smem + L::OFF_CTL);
    volatile int *abort_flag = &ctl->abort;
    const int warp = uniform(int(threadIdx.x >> 5)), lane = threadIdx.x & 31;
    const uint32_t sQ = base, sK = base + L::OFF_K, sV = base + L::OFF_V;

    // set-up that touches no memory of the launch before: barriers and tensor memory
    if (threadIdx.x == 0) {
        mbar_init(&ctl->q_ready, 2 * kRows);
        for (int s = 0; s < 2; ++s) {
            mbar_init(&ctl->k_full[s], 1);
            mbar_init(&ctl->k_empty[s], 2);  // both lanes (one tile: its block's lane, twice)
            mbar_init(&ctl->v_full[s], 1);
            mbar_init(&ctl->v_ready[s], 1);
            mbar_init(&ctl->v_empty[s], 2);
            for (int h = 0; h < 2; ++h) {
                mbar_init(&ctl->s_full[s][h], 1);
                mbar_init(&ctl->p_full[s][h], kRows / 32);
            }
            mbar_init(&ctl->o_done[s], 1);
        }
        mbar_init(&ctl->drain, 2);
        ctl->abort = 0;
        ctl->poisoned = 0;
        fence_mbarrier_init();
        fence_proxy_async_smem();
    }
    if (warp == W_MMA) {
        tmem_alloc(&ctl->tmem_base, kTmemCols);
        tmem_relinquish();
    }
    // the tables, q and the cache may be written by the kernel before this one
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // slot = tile * kv_heads * chunks + head * chunks + chunk: a tile's heads and chunks run together
    const unsigned per = unsigned(a.kv_heads) * unsigned(plan.chunks);
    const int slot = int(blockIdx.x / per), g = int(blockIdx.x % per) / plan.chunks, chunk = int(blockIdx.x % per) % plan.chunks;
    const int G = a.heads / a.kv_heads;
    int b = 0, row0 = 0;
    bool bad = false;
    const bool found = find_rows(a.batch, G, slot, b, row0, status);
    const SeqSpan sp = found ? seq_span(a.batch, b, bad) : SeqSpan{0, 0, 0};
    const KeyCut cut = cut_keys(sp, a.window, a.causal, plan.chunk);
    const int rows = min(kCtaRows, int(int64_t(sp.n) * G - row0));
    const RowSpan rs = rows > 0 ? rows_see(sp, row0 / G, (row0 + rows - 1) / G, a.window, a.causal) : RowSpan{0, 0, 0, 0};
    const bool whole = cut.chunks <= 1;
    const int64_t k0 = cut.base + int64_t(chunk) * plan.chunk;
    const int first = int(k0 > rs.lo ? k0 : rs.lo);                                      // keys [first, last)
    const int last = int(k0 + plan.chunk < rs.hi ? k0 + plan.chunk : int64_t(rs.hi));
    const bool none = cut.chunks == 0 || last <= first;
    const bool idle = !found || (none && !(whole && chunk == 0));  // (CTA-uniform: nothing to write)
    const int block0 = first / kBlock, nb = none || idle ? 0 : (last + kBlock - 1) / kBlock - block0;
    const int nt = rows > kRows ? 2 : 1;
    // lane w: steps 0 .. steps_of(w) - 1; step u is half u & 1 of block block_of(w, u)
    auto steps_of = [&](int w) { return nt == 2 ? 2 * nb : 2 * ((nb + 1 - w) >> 1); };
    auto block_of = [&](int w, int u) { return nt == 2 ? u >> 1 : (u & ~1) + w; };

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = uint32_t(uniform(int(ctl->tmem_base)));
    if (idle) {
        if (warp == W_MMA) tmem_dealloc(tmem, kTmemCols);
        return;
    }

    if (warp == W_K || warp == W_V) {
        // ---- copies of one plane (a warp each: K's slots and V's are freed at different times)
        const bool v = warp == W_V;
        const CUtensorMap *map = v ? &vmap : &kmap;
        uint64_t *const full = v ? ctl->v_full : ctl->k_full, *const empty = v ? ctl->v_empty : ctl->k_empty;
        const int nb_u = uniform(nb), g_u = uniform(g);
        BoxPages boxes(a, b, block0 * kBlock, kBlock, plan.box_rows, first, last);
        int issued = 0;
        for (; issued < nb_u; ++issued) {
            const int s = issued & 1, u = issued >> 1;
            boxes.seek(issued);
            if (u > 0 && !__all_sync(0xffffffffu, wait_phase(&empty[s], (u - 1) & 1, abort_flag, wait_ns, status))) break;
            const uint32_t dst = (v ? sV : sK) + uint32_t(s * L::TILE);
            const BoxRange br = boxes.range(issued);
            if (lane == 0) mbar_expect_tx(&full[s], uint32_t((br.hi - br.lo) * boxes.rows * 128 * L::HALVES));
            __syncwarp();
            boxes.each(issued, br, bad, [&](int row, int slot_in, int page) {
#pragma unroll
                for (int h = 0; h < L::HALVES; ++h)
                    tma_cache(dst + uint32_t(h * L::HALF + row * 128), map, 64 * h, g_u, slot_in, page, &full[s]);
            });
        }
        report_bad(bad, status);
        // every copy issued must land before the CTA exits
        if (lane == 0)
            for (int j = max(0, issued - 2); j < issued; ++j)
                mbar_wait_bounded(&full[j & 1], (j >> 1) & 1, drain_ns(wait_ns), status);
        __syncwarp();
    } else if (warp == W_MMA || warp == W_MMA + 1) {
        // ---- MMAs of lane w, by one thread
        const int w = warp - W_MMA;
        constexpr uint32_t type = is_half<T> ? 0u : (1u << 7) | (1u << 10);
        const int nb_u = uniform(nb), nt_u = uniform(nt), nd = uniform((a.dim + 15) / 16);  // nd: 16-feature steps that hold anything
        const uint32_t idesc_s = (1u << 4) | type | (uint32_t(kStep >> 3) << 17) | (uint32_t(kRows >> 4) << 24);
        const uint32_t idesc_o = (1u << 4) | type | (1u << 16) | (uint32_t(nd * 2) << 17) | (uint32_t(kRows >> 4) << 24);
        auto wait_on = [&](uint64_t *bar, uint32_t parity) { return wait_phase(bar, parity, abort_flag, wait_ns, status); };
        const int steps = nt_u == 2 ? 2 * nb_u : 2 * ((nb_u + 1 - w) >> 1);
        auto block_u = [&](int u) { return nt_u == 2 ? u >> 1 : (u & ~1) + w; };
        // uniform values and an elected lane: with values that the compiler takes for divergent, an MMA's issue took 100
        // cycles instead of the 48 (N = 64) or 64 that it runs for; offsets never carry out of a descriptor's address field
        const uint64_t dq = desc_k(sQ + uint32_t(nt_u == 2 ? w * L::TILE : 0));
        const uint64_t dk[2] = {desc_k(sK), desc_k(sK + L::TILE)};
        const uint64_t dv[2] = {desc_mn(sV, L::HALF), desc_mn(sV + L::TILE, L::HALF)};
        const uint32_t t_s = tmem + uint32_t(w * 128), t_o = tmem + kOCol + uint32_t(w * 128);
        auto issue_s = [&](int u) -> bool {
            const int j = block_u(u);
            if (!(u & 1) && !wait_on(&ctl->k_full[j & 1], (j >> 1) & 1)) return false;
            tc_fence_after();
            const uint64_t db = ((j & 1) ? dk[1] : dk[0]) + uint64_t((u & 1) * (kStep * 128 >> 4));
#pragma unroll
            for (int kk = 0; kk < DP / 16; ++kk) {
                const uint64_t off = uint64_t((((kk >> 2) * L::HALF) >> 4) + 2 * (kk & 3));
                if (kk < nd) tc_mma_f16(t_s + uint32_t((u & 1) * 64), dq + off, db + off, idesc_s, kk > 0);
            }
            tc_commit(&ctl->s_full[w][u & 1]);
            if (u & 1) {
                tc_commit(&ctl->k_empty[j & 1]);
                if (nt_u == 1) tc_commit(&ctl->k_empty[j & 1]);
            }
            return true;
        };
        if (elect_one()) {
            bool ok = steps == 0 || wait_on(&ctl->q_ready, 0);
            for (int u = 0; u < 2 && u < steps && ok; ++u) ok = issue_s(u);
            for (int u = 0; u < steps && ok; ++u) {
                const int j = block_u(u);
                ok = ((u & 1) || wait_on(&ctl->v_ready[j & 1], (j >> 1) & 1)) && wait_on(&ctl->p_full[w][u & 1], (u >> 1) & 1);
                if (!ok) break;
                tc_fence_after();
                const uint64_t db = ((j & 1) ? dv[1] : dv[0]) + uint64_t((u & 1) * (kStep * 128 >> 4));
                const uint32_t p = t_s + uint32_t((u & 1) * 64);
#pragma unroll
                for (int kk = 0; kk < kStep / 16; ++kk) {
                    const uint64_t bk = db + uint64_t(kk * 2048 >> 4);
                    mma_ts(t_o, p + uint32_t(kk * 8), bk, idesc_o, kk > 0 ? 1u : uint32_t(u > 0));
                    if constexpr (SPLIT_P) mma_ts(t_o, p + uint32_t(32 + kk * 8), bk, idesc_o, 1u);
                }
                tc_commit(&ctl->o_done[w]);
                if (u & 1) {
                    tc_commit(&ctl->v_empty[j & 1]);
                    if (nt_u == 1) tc_commit(&ctl->v_empty[j & 1]);
                }
                if (u + 2 < steps) ok = issue_s(u + 2);
            }
            tc_commit(&ctl->drain);  // when all of this thread's MMAs have ended
        }
        __syncwarp();
    } else if (warp == W_SOFT - 1) {
        // ---- V: slots that some row of the CTA must not multiply
        for (int j = 0; j < nb; ++j) {
            if (!__all_sync(0xffffffffu, wait_phase(&ctl->v_full[j & 1], (j >> 1) & 1, abort_flag, wait_ns, status))) break;
            const int key0 = (block0 + j) * kBlock;
            // rows [0, r0) and [r1, 128) of the block
            const int r0 = min(kBlock, max(0, max(first, rs.lo_all) - key0)), r1 = max(r0, min(kBlock, min(last, rs.hi_all) - key0));
            if (r0 > 0 || r1 < kBlock) {
                uint8_t *v = smem + L::OFF_V + (j & 1) * L::TILE;
                constexpr int CH = L::HALVES * 8;  // 16-byte pieces of a row
                for (int i = lane; i < (r0 + kBlock - r1) * CH; i += 32) {
                    const int x = i / CH, c = i % CH, r = x < r0 ? x : x - r0 + r1, key = key0 + r;
                    uint4 *p = reinterpret_cast<uint4 *>(v + (c >> 3) * L::HALF + r * 128 + (((c & 7) ^ (r & 7)) << 4));
                    if (key < first || key >= last) {
                        *p = make_uint4(0, 0, 0, 0);
                    } else {
                        uint4 w = *p;
                        if (any_nonfinite<T>(w)) {
                            take_nonfinite<T>(w, [](int, float) {});
                            *p = w;
                            ctl->poisoned = 1;  // (read behind the MMAs that follow v_ready)
                        }
                    }
                }
                fence_proxy_async_smem();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl->v_ready[j & 1]);
        }
    } else {
        // ---- softmax groups; first, both bring the rows of Q into the swizzled tiles
        const int w = (warp - W_SOFT) >> 2;
        {
            const uint32_t flip = a.scale < 0.f ? 0x80008000u : 0u;  // a negative scale turns q's sign
            const T *q = static_cast<const T *>(a.q) + int64_t(sp.q0) * a.q_token;
            // a group brings its tile, or half of the only one; all of a thread's loads are in flight together
            constexpr int CH = DP / 8, STEP = kRows / CH;  // 16-byte pieces of a row; rows between a thread's pieces
            const int tid = threadIdx.x & (kRows - 1), c = tid % CH;
            const int r_first = tid / CH + (nt == 2 ? 0 : w * (kRows / 2)), count = nt == 2 ? CH : CH / 2;
            const int row_from = row0 + (nt == 2 ? w * kRows : 0) + r_first;
            int i = row_from / G, hh = row_from % G;
            const int i_step = STEP / G, h_step = STEP % G;
            uint4 x[CH];
#pragma unroll
            for (int k = 0; k < CH; ++k) {
                x[k] = make_uint4(0, 0, 0, 0);
                if (k < count && row_from + k * STEP < row0 + rows && 8 * c < a.dim)
                    x[k] = *reinterpret_cast<const uint4 *>(q + int64_t(i) * a.q_token + int64_t(g * G + hh) * a.q_head + 8 * c);
                i += i_step;
                hh += h_step;
                if (hh >= G) {
                    hh -= G;
                    ++i;
                }
            }
#pragma unroll
            for (int k = 0; k < CH; ++k)
                if (k < count) {
                    const int r = r_first + k * STEP;
                    *reinterpret_cast<uint4 *>(smem + (nt == 2 ? w * L::TILE : 0) + (c >> 3) * L::HALF + r * 128 +
                                               (((c & 7) ^ (r & 7)) << 4)) =
                        make_uint4(x[k].x ^ flip, x[k].y ^ flip, x[k].z ^ flip, x[k].w ^ flip);
                }
            fence_proxy_async_smem();
            mbar_arrive(&ctl->q_ready);
        }
        const int r = (warp & 3) * 32 + lane;                        // row in the tile = TMEM lane
        const int row = (nt == 2 ? w * kRows : 0) + r;               // row of the CTA
        const uint32_t tl = uint32_t((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + tl + uint32_t(w * 128), to = tmem + tl + kOCol + uint32_t(w * 128);
        // scores stay unscaled; scale2 > 0 enters with the exponential (a zero scale as a tiny one, so that -inf stays)
        const float scale2 = fmaxf(fabsf(a.scale) * 1.4426950408889634f, 1e-30f);
        const KeyRange kr = row < rows ? keys_of(sp, (row0 + row) / G, a.window, a.causal) : KeyRange{0, INT32_MAX};  // (rows past the end: never written)
        const int lo = max(kr.lo, first), hi = min(kr.hi, last);
        const uint64_t scale22 = pair(scale2, scale2);
        float m = -INFINITY, l = 0.f;
        bool ok = true;
        const int done = steps_of(w);
        for (int u = 0; u < done; ++u) {
            ok = __all_sync(0xffffffffu, wait_phase(&ctl->s_full[w][u & 1], (u >> 1) & 1, abort_flag, wait_ns, status));
            if (!ok) break;
            tc_fence_after();
            const int key0 = (block0 + block_of(w, u)) * kBlock + (u & 1) * kStep;
            const int from = lo - key0, upto = hi - key0;  // this row's keys of the step: [from, upto)
            uint32_t va[32], vb[32];
            tm_ld32(ts + uint32_t((u & 1) * 64), va);
            tm_ld32(ts + uint32_t((u & 1) * 64 + 32), vb);
            tm_wait_ld(va);
            tm_wait_ld(vb);
            if (!__all_sync(0xffffffffu, from <= 0 && upto >= kStep)) {
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    if (i < from || i >= upto) va[i] = 0xff800000u;  // -inf
                    if (i + 32 < from || i + 32 >= upto) vb[i] = 0xff800000u;
                }
            }
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int i = 0; i < 32; ++i) mx[i & 3] = max3(mx[i & 3], __uint_as_float(va[i]), __uint_as_float(vb[i]));
            const float top = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]);
            const bool grow = top > m && (top - m) * scale2 > kLazy;
            const float mu = grow ? top : m;
            const float alpha = grow ? fast_ex2((m - mu) * scale2) : 1.f;
            const float neg = mu == -INFINITY ? 0.f : -mu * scale2;
            const uint64_t neg2 = pair(neg, neg);
            uint64_t sum2[2] = {pair(0.f, 0.f), pair(0.f, 0.f)};
            uint32_t hp[32], lp[SPLIT_P ? 32 : 1];
#pragma unroll
            for (int e = 0; e < 32; ++e) {  // keys 2e, 2e + 1 of the step
                const float s0 = __uint_as_float(e < 16 ? va[2 * e] : vb[2 * e - 32]);
                const float s1 = __uint_as_float(e < 16 ? va[2 * e + 1] : vb[2 * e - 31]);
                float d0, d1;
                unpair(fma2(pair(s0, s1), scale22, neg2), d0, d1);
                const float p0 = fast_ex2(d0), p1 = fast_ex2(d1);
                sum2[e & 1] = add2(sum2[e & 1], pair(p0, p1));
                // the weights in the cache's type (one type for both operands); an f32 output keeps the remainder
                hp[e] = pack16<T>(p0, p1);
                if constexpr (SPLIT_P) {
                    float h0, h1;
                    unpack16<T>(hp[e], h0, h1);
                    lp[e] = pack16<T>(p0 - h0, p1 - h1);
                }
            }
            tm_st32(ts + uint32_t((u & 1) * 64), hp);
            if constexpr (SPLIT_P) tm_st32(ts + uint32_t((u & 1) * 64 + 32), lp);
            if (u > 0 && __any_sync(0xffffffffu, grow)) {
                // rescale this row of O (rows that keep m by 1) once the step before has accumulated into it
                ok = __all_sync(0xffffffffu, wait_phase(&ctl->o_done[w], (u - 1) & 1, abort_flag, wait_ns, status));
                if (!ok) break;
                tc_fence_after();
#pragma unroll 1
                for (int c = 0; c < (a.dim + 31) / 32; ++c) {
                    uint32_t o[32];
                    tm_ld32(to + uint32_t(c * 32), o);
                    tm_wait_ld(o);
#pragma unroll
                    for (int q = 0; q < 32; ++q) o[q] = __float_as_uint(__uint_as_float(o[q]) * alpha);
                    tm_st32(to + uint32_t(c * 32), o);
                }
            }
            tm_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl->p_full[w][u & 1]);
            float s0, s1;
            unpair(add2(sum2[0], sum2[1]), s0, s1);
            l = l * alpha + (s0 + s1);
            m = mu;
        }
        if (ok && done > 0) {
            // (a lane has an even number of steps; the last one's S told that P V up to step done - 3 has ended, and a
            // parity tells a phase only from its neighbours)
            ok = __all_sync(0xffffffffu, wait_phase(&ctl->o_done[w], (done - 2) & 1, abort_flag, wait_ns, status) &&
                                             wait_phase(&ctl->o_done[w], (done - 1) & 1, abort_flag, wait_ns, status));
            tc_fence_after();
        }
        // one tile: group 1's rows go to group 0 through shared memory (over Q and K, which no MMA reads any more:
        // both groups have seen their last MMA end)
        float *ex = reinterpret_cast<float *>(smem);
        float *exm = reinterpret_cast<float *>(smem + L::OFF_ML), *exl = exm + kRows;
        float scale_own = 1.f, scale_other = 0.f;
        if (nt == 1) {
            asm volatile("bar.sync 1, 256;" ::: "memory");
            ok = ok && *abort_flag == 0;
            if (w == 1) {
                exm[r] = m;
                exl[r] = l;
                if (ok && done > 0) {
#pragma unroll 1
                    for (int c = 0; c < (a.dim + 31) / 32; ++c) {
                        uint32_t o[32];
                        tm_ld32(to + uint32_t(c * 32), o);
                        tm_wait_ld(o);
#pragma unroll
                        for (int i = 0; i < 32; i += 4)
                            *reinterpret_cast<uint4 *>(&ex[r * L::MPAD + c * 32 + i]) = make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                    }
                }
            }
            asm volatile("bar.sync 1, 256;" ::: "memory");
            if (w == 0 && nb > 1) {
                const float mo = exm[r], top = fmaxf(m, mo);  // (m == top holds where both are -inf)
                scale_own = m == top ? 1.f : fast_ex2((m - top) * scale2);
                scale_other = mo == top ? 1.f : fast_ex2((mo - top) * scale2);
                l = l * scale_own + exl[r] * scale_other;
                m = top;
            }
        }
        auto to_cols = [&](int c) { return to + uint32_t(c * 32); };
        // values that are not finite, of keys that this row sees and another row of the CTA does not (columns 32 c ..)
        auto add_hidden = [&](int c, uint32_t (&o)[32]) {
            for (int key = lo; key < hi; ++key) {
                if (key >= rs.lo_all && key < rs.hi_all) {
                    key = rs.hi_all - 1;
                    continue;
                }
                const int entry = key / a.batch.page_size;
                bool ignore = false;
                const int64_t p = page_of(a.batch, b, entry, ignore);
                const T *v = static_cast<const T *>(a.v) + (p < 0 ? 0 : p) * a.page_stride +
                             int64_t(key - entry * a.batch.page_size) * a.slot_stride + int64_t(g) * a.head_stride + c * 32;
#pragma unroll 1
                for (int i = 0; i < 32 && c * 32 + i < a.dim; ++i) {
                    const float x = float(v[i]);
                    if (!isfinite(x))
#pragma unroll
                        for (int e = 0; e < 32; ++e)  // (o stays in registers)
                            if (e == i) o[e] = __float_as_uint(__uint_as_float(o[e]) + x);
                }
            }
        };
        if (ok && (nt == 2 || w == 0)) {
            const int64_t t = int64_t(sp.q0) + (row0 + row) / G;
            const int h = g * G + (row0 + row) % G;
            const bool mine = row < rows;
            const float inv = whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;  // no key: zeros
            if (!whole && mine) part_ml[partial_at(a, chunk, t, h)] = make_float2(m == -INFINITY ? m : m * scale2, l);
            const bool poisoned = *reinterpret_cast<volatile int *>(&ctl->poisoned) != 0;
            // Rows leave through shared memory, 128 bytes of each at a time, so that eight lanes store one row's piece.
            // A warp's 4 KB lie over the lane's Q tile, which its last MMA has left; with one tile (whose Q the other
            // group's exchange lies over) over V, which nothing reads any more.
            uint8_t *stage = smem + (nt == 2 ? w * L::TILE : L::OFF_V) + (warp & 3) * 4096;
            auto put = [&](bool partial, auto *to, int64_t t_stride, int64_t h_stride) {
                using E = typename std::remove_pointer<decltype(to)>::type;
                constexpr int W = 128 / sizeof(E);  // columns of a piece: 32 in f32, 64 in 16 bits
                int64_t at[8];                      // where the rows that this lane stores a part of go
                const int r_out = row - lane + (lane >> 3);
                int i = (row0 + r_out) / G, hh = (row0 + r_out) % G;
                const int i_step = 4 / G, h_step = 4 % G;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int64_t tt = int64_t(sp.q0) + i;
                    at[k] = partial ? partial_at(a, chunk, tt, g * G + hh) * a.dim : tt * t_stride + int64_t(g * G + hh) * h_stride;
                    i += i_step;
                    hh += h_step;
                    if (hh >= G) {
                        hh -= G;
                        ++i;
                    }
                }
                for (int c0 = 0; c0 < a.dim; c0 += W) {
#pragma unroll
                    for (int part = 0; part < W / 32; ++part) {
                        const int c = c0 / 32 + part;
                        uint32_t o[32];
                        if (nb > 0) {
                            tm_ld32(to_cols(c), o);
                            tm_wait_ld(o);
                        }
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            float x = nb > 0 ? __uint_as_float(o[i]) : 0.f;
                            if (nt == 1 && nb > 1) x = x * scale_own + ex[r * L::MPAD + c * 32 + i] * scale_other;
                            o[i] = __float_as_uint(x);
                        }
                        if (poisoned && mine) add_hidden(c, o);
#pragma unroll
                        for (int i = 0; i < 32; i += 16 / int(sizeof(E))) {
                            uint4 v;
                            auto f = [&](int e) { return __uint_as_float(o[i + e]) * inv; };
                            if constexpr (sizeof(E) == 4)
                                v = make_uint4(__float_as_uint(f(0)), __float_as_uint(f(1)), __float_as_uint(f(2)), __float_as_uint(f(3)));
                            else
                                v = make_uint4(pack16<E>(f(0), f(1)), pack16<E>(f(2), f(3)), pack16<E>(f(4), f(5)), pack16<E>(f(6), f(7)));
                            const int piece = (part * 32 + i) * int(sizeof(E)) / 16;
                            *reinterpret_cast<uint4 *>(stage + lane * 128 + ((piece ^ (lane & 7)) << 4)) = v;
                        }
                    }
                    __syncwarp();
                    const int piece = lane & 7, col = c0 + piece * (16 / int(sizeof(E)));
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const int rr = k * 4 + (lane >> 3);
                        const uint4 v = *reinterpret_cast<const uint4 *>(stage + rr * 128 + ((piece ^ (rr & 7)) << 4));
                        if (r_out + 4 * k < rows && col < a.dim) *reinterpret_cast<uint4 *>(to + at[k] + col) = v;
                    }
                    __syncwarp();
                }
            };
            if (whole) put(false, static_cast<TO *>(a.out), a.out_token, a.out_head);
            else put(true, part_o, 0, 0);
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

// CTA slots of row tiles, at most: each sequence leaves less than one tile unfilled.
int64_t tile_bound(int64_t group, int64_t seqs, int64_t tokens) {
    return (tokens * group + std::min(seqs, tokens) * (kCtaRows - 1)) / kCtaRows;
}

// The most chunks worth having: four turns of every SM.
int64_t split_bound(int64_t ctas, int64_t max_kv) {
    const int64_t blocks = (max_kv + kBlock - 1) / kBlock;
    return std::max<int64_t>(1, std::min({(4 * kNumSms + ctas - 1) / ctas, (blocks + kMinBlocks - 1) / kMinBlocks,
                                          int64_t(kMaxSplits)}));
}

// Chunks of keys: the number for which turns of the SMs x (blocks a CTA + the
// cost of a CTA's start and end, in blocks) is least.
KeyPlan chunk_plan(int64_t ctas, int64_t max_q, int64_t max_kv, int64_t window, int page_size) {
    KeyPlan p = {};
    const int64_t span = key_span(max_q, max_kv, window), blocks = std::max<int64_t>(1, (span + kBlock - 1) / kBlock);
    int64_t best = 1;
    double least = 0;
    for (int64_t s = 1; s <= split_bound(ctas, span); ++s) {
        const double turns = double((ctas * s + kNumSms - 1) / kNumSms);
        const double cost = turns * (double((blocks + s - 1) / s) + (s > 1 ? 4.5 : 3.0)) + (s > 1 ? 2.0 : 0.0);
        if (s == 1 || cost < least) {
            best = s;
            least = cost;
        }
    }
    p.chunk = int((blocks + best - 1) / best * kBlock);
    p.chunks = int((blocks * kBlock + p.chunk - 1) / p.chunk);
    p.box_rows = std::min(page_size & -page_size, kBlock);
    return p;
}

template <typename T, typename TO, int DP>
cudaError_t launch_chunk(const PagedArgs &a, void *ws, const LaunchCtx &ctx) {
    using L = ChunkLayout<DP>;
    const int64_t tiles = tile_bound(a.heads / a.kv_heads, a.batch.seqs, a.batch.tokens);
    const KeyPlan plan = chunk_plan(tiles * a.kv_heads, a.batch.max_q, a.batch.max_kv, a.window, a.batch.page_size);
    const int64_t ctas = tiles * a.kv_heads * plan.chunks;
    if (ctas > INT32_MAX) return cudaErrorInvalidValue;
    CUtensorMap km, vm;
    cudaError_t e = cache_maps<T>(a, plan.box_rows, &km, &vm);
    if (e != cudaSuccess) return e;
    auto kernel = paged_chunk_kernel<T, TO, DP>;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::BYTES);
    if (e != cudaSuccess) return e;
    float *po = static_cast<float *>(ws);
    float2 *pml = reinterpret_cast<float2 *>(po + int64_t(plan.chunks) * a.batch.tokens * a.heads * a.dim);
    e = launch_dependent(kernel, dim3(unsigned(ctas)), kThreads, L::BYTES, ctx.stream, km, vm, a, plan, po, pml, ctx.status,
                         ctx.wait_ns);
    if (e != cudaSuccess || plan.chunks == 1) return e;
    return launch_join<TO>(a, plan, po, pml, ctx);
}

template <typename T, typename TO>
cudaError_t launch_chunk_io(const PagedArgs &a, void *ws, const LaunchCtx &ctx) {
    return a.dim <= 64 ? launch_chunk<T, TO, 64>(a, ws, ctx) : launch_chunk<T, TO, 128>(a, ws, ctx);
}

}  // namespace

int64_t attention_paged_chunk_bound(int64_t heads, int64_t kv_heads, int64_t seqs, int64_t tokens, int64_t max_kv) {
    return split_bound(tile_bound(heads / kv_heads, seqs, tokens) * kv_heads, max_kv);
}

cudaError_t launch_attention_paged_chunk(const PagedArgs &a, int dtype, bool out_f32, void *ws, const LaunchCtx &ctx) {
    if (dtype == TQ2_F16) {
        if (out_f32) return launch_chunk_io<__half, float>(a, ws, ctx);
        return launch_chunk_io<__half, __half>(a, ws, ctx);
    }
    if (out_f32) return launch_chunk_io<__nv_bfloat16, float>(a, ws, ctx);
    return launch_chunk_io<__nv_bfloat16, __nv_bfloat16>(a, ws, ctx);
}

}  // namespace tq2
