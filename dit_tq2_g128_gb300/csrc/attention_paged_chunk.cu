// Attention of a step's new tokens over a paged key/value cache: many query rows
// per (sequence, key head), on the tcgen05 tensor cores.
//
// Mathematics: the online softmax of attention_paged.cu with the query rows in M.
// The rows of a sequence and key head are its new tokens times the query heads of
// the group, row = token * G + head, so a 128-row tile of a chunk reads each key
// for all G heads at once.
//
//  * An item is up to 256 consecutive rows (two tiles) of one (sequence, key head).
//    Where the items fill the SMs they stay whole, a CTA of the grid for each, a
//    sequence's longest first; a CTA near its item's end takes over one that has not started
//    (a cluster launch control request), so that copies, lookups and set-up of the next item run
//    under this one's end: 8 us between items became 6 (one prompt of 4096 tokens 117 -> 107
//    us, 16 of 512 101 -> 86, ragged prompts 242 -> 227).  Where they are few and long their
//    blocks of 128 keys, in one line with the cost of an item's start
//    and end, are cut into as many equal runs as there are SMs, and a CTA takes a run: it
//    starts once, copies ahead into its next item, and its next Q comes as soon as the
//    last S that reads the old one has ended; pieces of a cut item go to the workspace
//    and a second, dependent launch joins them in order.  (The rule and both sides'
//    times: chunk_launch.)
//  * Warps 0 and 12 copy K and V through two-stage rings by paged tensor copies (boxes
//    of rows inside one page), warp 0 Q too; warps 1 and 2 issue the MMAs of lane 0 and
//    1 (below); warp 3 looks after V; warps 4-7 and 8-11 are the lanes' softmax groups,
//    one thread per row (= tensor-memory lane).  Warp 13 claims whole items.
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
//    weights' remainder follows as a second term in the other 32 (errors of 1.5e-6 of
//    the result in binary16 and 2.5e-6 in bf16 at 500 keys; a third bf16 term, through
//    shared memory, made that 1.5e-6 and the kernel 30 % slower).  binary16 weights are
//    lifted first (weight_lift).
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
constexpr int kThreads = 448;
constexpr int kClaimAhead = 4;  // blocks before an item's end at which the CTA asks for its next one
// An item's start and end, in blocks, for the shares of cut items (512 tokens over 32768 keys, and ragged prompts if cut:
// 2 took 207 and 277 us, 4 207 and 248, 8 213 and 271 when measured, the former 195 since).
constexpr int kStartUnits = 4;
constexpr int kMinUnits = 4;    // units of a run, at least, where items may be cut
constexpr int kJoinRows = 4;    // rows of a warp of the join
constexpr int kJoinParts = kCtaRows / (kJoinRows * kJoinWarps);  // its blocks per cut item
constexpr uint32_t kTmemCols = 512, kOCol = 256;
constexpr float kLazy = 8.f;    // log2 growth of the maximum that O is rescaled for
constexpr int W_K = 0, W_MMA = 1, W_SOFT = 4, W_V = 12, W_CLAIM = 13;  // W_MMA + lane; warp 3 looks after V

template <int DP>
struct ChunkLayout {
    static constexpr int HALVES = DP / 64;
    static constexpr int HALF = 128 * 128;            // 128 rows x 64 features, swizzled
    static constexpr int TILE = HALF * HALVES;        // Q tile, K block, V block
    static constexpr int OFF_K = 2 * TILE, OFF_V = OFF_K + 2 * TILE;
    static constexpr int OFF_STAGE = OFF_V + 2 * TILE; // 4 KB a softmax warp, for rows on their way out
    static constexpr int OFF_CTL = OFF_STAGE + 8 * 4096;
    static constexpr int BYTES = OFF_CTL + 512 + 1024;
    static_assert(BYTES <= 232448, "shared memory budget");
};

// An item of a prompt: rows from row0 on of a sequence (its first token, its new tokens, its keys) and a key head; left:
// 1, or 0 where there is none.
struct alignas(16) Item {
    int b, row0, g, left, q0, n, kv, unused;
};

struct ChunkCtl {
    uint4 answer;            // to the request for another CTA's item
    Item next[3];            // whole items: the first in [2], those after it in [0] and [1] in turn
    uint64_t answered, want, item_full[2], item_free[2];
    uint64_t q_ready, q_free, k_full[2], k_empty[2], v_full[2], v_ready[2], v_empty[2];
    uint64_t s_full[2][2], p_full[2][2], o_done[2], drain;  // [lane][step & 1]
    uint64_t item_done[2];   // a lane's last P V of an item has ended
    uint32_t tmem_base;
    int abort;
    int poisoned[4];         // by item (of those with blocks, from 1 on) modulo 4: the last whose V had values taken out
    int item;                // the item that q_ready announces: twice its blocks, one more for two tiles; 0: the run is over
    int soft_go[2];          // the softmax groups go on with next[.]
    int b, row0, g, u, left; // where this CTA's run begins: sequence, rows, key head, unit; its units
};
static_assert(sizeof(ChunkCtl) <= 512, "control block");

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

__device__ __forceinline__ void groups_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }  // both softmax groups

// A wait as wait_phase's for what takes an item's time: it leaves the schedulers alone.
__device__ __forceinline__ bool doze_phase(uint64_t *bar, uint32_t parity, volatile int *abort_flag, uint64_t wait_ns, unsigned int *status) {
    const uint32_t addr = smem_u32(bar);
    const uint64_t t0 = globaltimer_ns();
    for (;;) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(addr), "r"(parity)
            : "memory");
        if (ok) return true;
        if (*abort_flag) return false;
        if (globaltimer_ns() - t0 >= wait_ns) {
            atomicOr(status, static_cast<unsigned int>(TQ2_ERR_TIMEOUT));
            *abort_flag = 1;
            return false;
        }
        __nanosleep(500);
    }
}

// Asks for a CTA of this grid that has not started, to be done here in its place; the answer comes by bulk copy.
__device__ __forceinline__ void request_cta(uint4 *answer, uint64_t *bar) {
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                     smem_u32(answer)),
                 "r"(smem_u32(bar))
                 : "memory");
}
// Its index, or -1: there is none left (no request may follow).
__device__ __forceinline__ int requested_cta(const uint4 *answer) {
    uint32_t got, x;
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b128 h;\n\t"
        "ld.shared.b128 h, [%2];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t"
        "mov.u32 %1, 0;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, h;\n\t}"
        : "=r"(got), "=r"(x)
        : "r"(smem_u32(answer))
        : "memory");
    return got ? int(x) : -1;
}

// 64 features of a tile's rows of Q: feature x, head, token
__device__ __forceinline__ void tma_rows(uint32_t dst, const CUtensorMap *map, int x, int head, int token, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(head), "r"(token), "r"(smem_u32(bar))
        : "memory");
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

// How a call is shared out: the rows of a copy, whether items may be cut, and whether
// Q's tiles are copied by tensor copies (the group divides a tile, the scale is not
// negative).
struct ChunkPlan {
    int box_rows;
    int split;
    int q_copies;
};

// What a cut item's piece says to the join: sequence + 1 (0: no piece), first row, key
// head, 1 if the item's last key is in it.
using Piece = int4;

__device__ __forceinline__ int tiles_in(const SeqSpan &sp, int G) { return int((int64_t(sp.n) * G + kCtaRows - 1) / kCtaRows); }

__device__ __forceinline__ ItemSpan item_of(const PagedArgs &a, const SeqSpan &sp, int row0) {
    return item_span(sp, a.heads / a.kv_heads, row0, kCtaRows, a.window, a.causal, kBlock);
}

// Items in the order of a grid that takes them whole (one warp): from the last sequence's last tile (the longest of a
// prompt) on, key heads innermost.  Successive indices mostly rise: the search goes on from where it stands.
struct ItemFinder {
    const PagedArgs &a;
    const int G;
    int top, passed;  // sequences below top are left; the others' items

    __device__ __forceinline__ explicit ItemFinder(const PagedArgs &args) : a(args), G(args.heads / args.kv_heads), top(args.batch.seqs), passed(0) {}
    __device__ __forceinline__ Item find(int index, unsigned int *status) {
        const BatchView &bt = a.batch;
        const int lane = threadIdx.x & 31;
        if (index < passed) {
            top = bt.seqs;
            passed = 0;
        }
        for (; top > 0; top -= 32) {
            const int b = top - 1 - lane;
            SeqSpan sp{0, 0, 0};
            if (b >= 0) {
                bool bad = false;
                sp = seq_span(bt, b, bad);
                report_bad(bad, status);
            }
            const int tiles = tiles_in(sp, G);
            int upto = tiles * a.kv_heads;  // inclusive over the lanes
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, upto, d);
                if (lane >= d) upto += x;
            }
            const unsigned hit = __ballot_sync(0xffffffffu, index - passed < upto);
            if (hit) {
                const int l = __ffs(hit) - 1, at = index - passed - __shfl_sync(0xffffffffu, upto - tiles * a.kv_heads, l);
                return Item{top - 1 - l, (__shfl_sync(0xffffffffu, tiles, l) - 1 - at / a.kv_heads) * kCtaRows, at % a.kv_heads, 1,
                            __shfl_sync(0xffffffffu, sp.q0, l), __shfl_sync(0xffffffffu, sp.n, l), __shfl_sync(0xffffffffu, sp.kv, l), 0};
            }
            passed += __shfl_sync(0xffffffffu, upto, 31);
        }
        return Item{0, 0, 0, 0, 0, 0, 0, 0};
    }
};

// The run of this CTA (one warp): `left` units from unit u of item (b, row0, g) on.
template <bool SPLIT>
__device__ __forceinline__ void find_run(const PagedArgs &a, ChunkCtl *ctl, unsigned int *status) {
    const BatchView &bt = a.batch;
    const int lane = threadIdx.x & 31, G = a.heads / a.kv_heads;
    if (!SPLIT) {  // item blockIdx.x of all
        const Item it = ItemFinder(a).find(int(blockIdx.x), status);
        if (lane == 0) {
            ctl->b = it.b;
            ctl->row0 = it.row0;
            ctl->g = it.g;
            ctl->u = 0;
            ctl->left = it.left;
            ctl->next[2] = it;
        }
        return;
    }
    auto weight = [&](const SeqSpan &sp, int tile) { return kStartUnits + max(1, item_of(a, sp, tile * kCtaRows).blocks); };
    // units of sequences base + lane, of one key head
    auto units_of = [&](int base) {
        SeqSpan sp{0, 0, 0};
        if (base + lane < bt.seqs) {
            bool bad = false;
            sp = seq_span(bt, base + lane, bad);
            report_bad(bad, status);
        }
        const int tiles = tiles_in(sp, G);
        int units = 0;
        if (__reduce_max_sync(0xffffffffu, unsigned(tiles)) <= 4) {
            for (int t = 0; t < tiles; ++t) units += weight(sp, t);
        } else {  // long prompts: a sequence's tiles over the lanes
            for (int l = 0; l < 32 && base + l < bt.seqs; ++l) {
                const SeqSpan x{__shfl_sync(0xffffffffu, sp.q0, l), __shfl_sync(0xffffffffu, sp.n, l), __shfl_sync(0xffffffffu, sp.kv, l)};
                const int n = tiles_in(x, G);
                int sum = 0;
                for (int t = lane; t < n; t += 32) sum += weight(x, t);
                sum = int(__reduce_add_sync(0xffffffffu, unsigned(sum)));
                if (lane == l) units = sum;
            }
        }
        return units;
    };
    // The host has checked that the units of the step's tokens fit 32 bits; sequences of a bad batch that claim the same
    // tokens may pass that, and then nothing is done.
    auto sum_of = [](int units) {
        return (int64_t(__reduce_add_sync(0xffffffffu, unsigned(units) >> 16)) << 16) +
               __reduce_add_sync(0xffffffffu, unsigned(units) & 0xffffu);
    };
    const int head = units_of(0);
    int64_t sum = sum_of(head);
    for (int base = 32; base < bt.seqs; base += 32) sum += sum_of(units_of(base));
    sum *= a.kv_heads;
    if (sum > INT32_MAX - kNumSms) {
        if (lane == 0) {
            report_bad(true, status);
            ctl->left = 0;
        }
        return;
    }
    const int total = int(sum);
    const int ctas = int(gridDim.x), share = max(kMinUnits, (total + ctas - 1) / ctas);
    const int64_t start = int64_t(blockIdx.x) * share;
    if (lane == 0) ctl->left = start < total ? int(min(int64_t(share), total - start)) : 0;
    if (start >= total) return;
    int from = int(start);  // units left to pass
    for (int base = 0; base < bt.seqs; base += 32) {
        const int units = (base == 0 ? head : units_of(base)) * a.kv_heads;
        int upto = units;  // inclusive over the lanes
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, upto, d);
            if (lane >= d) upto += x;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, from < upto);
        if (!hit) {
            from -= __shfl_sync(0xffffffffu, upto, 31);
            continue;
        }
        const int l = __ffs(hit) - 1, b = base + l;
        from -= __shfl_sync(0xffffffffu, upto - units, l);
        bool ignore = false;
        const SeqSpan sp = seq_span(bt, b, ignore);
        const int tiles = tiles_in(sp, G);
        for (int t0 = 0; t0 < tiles; t0 += 32) {
            const int w = t0 + lane < tiles ? weight(sp, t0 + lane) : 0;
            int sum = w * a.kv_heads;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, sum, d);
                if (lane >= d) sum += x;
            }
            const unsigned found = __ballot_sync(0xffffffffu, from < sum);
            if (found) {
                if (lane == __ffs(found) - 1) {
                    const int at = from - (sum - w * a.kv_heads);
                    ctl->b = b;
                    ctl->row0 = (t0 + lane) * kCtaRows;
                    ctl->g = at / w;
                    ctl->u = at % w;
                }
                return;
            }
            from -= __shfl_sync(0xffffffffu, sum, 31);
        }
        return;
    }
}

// A CTA's run of cut items, or a whole item, part by part: every role walks it by itself (whole warps).
struct ChunkWalk {
    const PagedArgs &a;
    const ChunkPlan &plan;
    const int G;
    int b, row0, g, u, left;
    SeqSpan sp;
    ItemSpan it;
    int units, take;
    // the current item's part: rows, lanes' tiles, blocks from block0 on, keys [first, last)
    int rows, nt, block0, nb, first, last;

    __device__ __forceinline__ ChunkWalk(const PagedArgs &args, const ChunkPlan &p, const ChunkCtl *ctl)
        : a(args), plan(p), G(args.heads / args.kv_heads), b(uniform(ctl->b)), row0(uniform(ctl->row0)), g(uniform(ctl->g)),
          u(uniform(ctl->u)), left(uniform(ctl->left)) {
        if (left > 0) {
            load();
            tile();
        }
    }
    __device__ __forceinline__ void load() {
        bool ignore = false;
        const SeqSpan s = seq_span(a.batch, b, ignore);  // (reported by find_run)
        sp = SeqSpan{uniform(s.q0), uniform(s.n), uniform(s.kv)};
    }
    // another whole item
    __device__ __forceinline__ void begin(const Item *next) {
        b = uniform(next->b);
        row0 = uniform(next->row0);
        g = uniform(next->g);
        u = 0;
        left = uniform(next->left);
        sp = SeqSpan{uniform(next->q0), uniform(next->n), uniform(next->kv)};
        if (left > 0) tile();
    }
    __device__ __forceinline__ void tile() {
        it = item_of(a, sp, row0);
        units = plan.split ? kStartUnits + max(1, it.blocks) : 1;
    }
    __device__ __forceinline__ bool more() {
        if (left <= 0) return false;
        take = min(left, units - u);
        // unit kStartUnits + k is block k
        const int k0 = plan.split ? max(0, u - kStartUnits) : 0;
        const int k1 = plan.split ? min(it.blocks, max(0, u + take - kStartUnits)) : it.blocks;
        rows = it.rows;
        nt = rows > kRows ? 2 : 1;
        block0 = it.block0 + k0;
        nb = max(0, k1 - k0);
        first = max(it.see.lo, block0 * kBlock);
        last = min(it.see.hi, (block0 + nb) * kBlock);
        return true;
    }
    __device__ __forceinline__ bool begins() const { return u <= kStartUnits; }  // its first block (and something of it)
    __device__ __forceinline__ bool whole() const { return nb == it.blocks; }
    // nothing of this item falls to this run (only a part of its start does)
    __device__ __forceinline__ bool skip() const { return nb == 0 && !(it.blocks == 0 && u + take == units); }
    // where a cut item's piece goes: a run's first piece, begun by the run before, or its last
    __device__ __forceinline__ int slot() const { return 2 * int(blockIdx.x) + begins(); }
    __device__ __forceinline__ int steps(int w) const { return nt == 2 ? 2 * nb : 2 * ((nb + 1 - w) >> 1); }
    // step s of lane w is half s & 1 of block:
    __device__ __forceinline__ int block(int w, int s) const { return nt == 2 ? s >> 1 : (s & ~1) + w; }
    __device__ __forceinline__ void next() {
        left -= take;
        u += take;
        if (u < units) return;
        u = 0;
        if (++g < a.kv_heads || left <= 0) return;
        g = 0;
        row0 += kCtaRows;
        if (int64_t(row0) >= int64_t(sp.n) * G) {
            row0 = 0;
            while (++b < a.batch.seqs) {
                load();
                if (sp.n > 0) break;
            }
        }
        tile();
    }
};

template <bool B>
struct bool_c {
    static constexpr bool value = B;
};

template <typename T, typename TO, int DP, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
paged_chunk_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                   const __grid_constant__ CUtensorMap qmap, const PagedArgs a, const ChunkPlan plan,
                   float *__restrict__ part_o, float2 *__restrict__ part_ml, Piece *__restrict__ pieces, unsigned int *status,
                   uint64_t wait_ns) {
    using L = ChunkLayout<DP>;
    constexpr bool SPLIT_P = sizeof(TO) == 4;
    extern __shared__ uint8_t chunk_raw[];
    const uint32_t raw = smem_u32(chunk_raw), pad = (1024u - (raw & 1023u)) & 1023u, base = raw + pad;
    uint8_t *smem = chunk_raw + pad;
    ChunkCtl *ctl = reinterpret_cast<ChunkCtl *>(smem + L::OFF_CTL);
    volatile int *abort_flag = &ctl->abort;
    const int warp = uniform(int(threadIdx.x >> 5)), lane = threadIdx.x & 31;
    const int G = a.heads / a.kv_heads;
    const uint32_t sQ = base, sK = base + L::OFF_K, sV = base + L::OFF_V;

    // set-up that touches no memory of the launch before: barriers and tensor memory
    if (threadIdx.x == 0) {
        mbar_init(&ctl->q_ready, 1);
        mbar_init(&ctl->q_free, 2);
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
            mbar_init(&ctl->item_done[s], 1);
        }
        mbar_init(&ctl->drain, 2);
        mbar_init(&ctl->answered, 1);
        mbar_init(&ctl->want, 1);
        for (int s = 0; s < 2; ++s) {
            mbar_init(&ctl->item_full[s], 1);
            mbar_init(&ctl->item_free[s], 2 + 1 + 2 * kRows / 32);  // K's, V's and V's second warp, the softmax groups
        }
        ctl->abort = 0;
        for (int &p : ctl->poisoned) p = 0;
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
    if (warp == 0) {
        find_run<SPLIT>(a, ctl, status);
        if (lane < 2 && pieces) pieces[2 * blockIdx.x + lane] = make_int4(0, 0, 0, 0);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = uint32_t(uniform(int(ctl->tmem_base)));
    ChunkWalk walk(a, plan, ctl);
    // Counters that run on over the items: blocks copied (slot = parity), this lane's steps (even an item), and the
    // items that have blocks (Q's phases).
    int blocks = 0, qi = 0, claims = 0;
    // The item after the current one, for the roles of one warp: of the run, or as the claiming warp says.
    auto next_item = [&](bool &ok) {
        walk.next();
        if constexpr (!SPLIT) {
            if (!ok) return;
            const int slot = claims & 1;
            ok = __all_sync(0xffffffffu, wait_phase(&ctl->item_full[slot], (claims >> 1) & 1, abort_flag, wait_ns, status));
            if (!ok) return;
            walk.begin(&ctl->next[slot]);
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl->item_free[slot]);
            ++claims;
        }
    };

    if (warp == W_K || warp == W_V) {
        // ---- copies of one plane (a warp each: K's slots and V's are freed at different times), and Q by K's warp
        const bool v = warp == W_V;
        const CUtensorMap *map = v ? &vmap : &kmap;
        uint64_t *const full = v ? ctl->v_full : ctl->k_full, *const empty = v ? ctl->v_empty : ctl->k_empty;
        bool bad = false, ok = true;
        for (; ok && walk.more(); next_item(ok)) {
            const int claim = !v && !SPLIT ? max(0, walk.nb - kClaimAhead) : -1;
            if (walk.nb == 0) {
                if (claim == 0 && lane == 0) mbar_arrive(&ctl->want);
                continue;
            }
            const int nb = uniform(walk.nb), g = uniform(walk.g), nt = uniform(walk.nt);
            const int q_token = uniform(walk.sp.q0 + walk.row0 / G);
            if (!v && plan.q_copies) {
                if (qi > 0) ok = __all_sync(0xffffffffu, wait_phase(&ctl->q_free, (qi - 1) & 1, abort_flag, wait_ns, status));
                if (!ok) break;
                if (elect_one()) {
                    *reinterpret_cast<volatile int *>(&ctl->item) = 2 * nb + (nt == 2);
                    mbar_expect_tx(&ctl->q_ready, uint32_t(nt * L::TILE));
                    for (int t = 0; t < nt; ++t)
#pragma unroll
                        for (int h = 0; h < L::HALVES; ++h)
                            tma_rows(sQ + uint32_t(t * L::TILE + h * L::HALF), &qmap, 64 * h, g * G, q_token + t * (kRows / G),
                                     &ctl->q_ready);
                }
                __syncwarp();
            }
            ++qi;
            BoxPages boxes(a, walk.b, walk.block0 * kBlock, kBlock, plan.box_rows, walk.first, walk.last);
            blocks = uniform(blocks);
            for (int j = 0; j < nb; ++j, ++blocks) {
                const int s = blocks & 1, u = blocks >> 1;
                boxes.seek(j);
                if (j == claim && lane == 0) mbar_arrive(&ctl->want);
                if (u > 0) ok = __all_sync(0xffffffffu, wait_phase(&empty[s], (u - 1) & 1, abort_flag, wait_ns, status));
                if (!ok) break;
                const uint32_t dst = (v ? sV : sK) + uint32_t(s * L::TILE);
                const BoxRange br = boxes.range(j);
                if (lane == 0) mbar_expect_tx(&full[s], uint32_t((br.hi - br.lo) * boxes.rows * 128 * L::HALVES));
                __syncwarp();
                boxes.each(j, br, bad, [&](int row, int slot_in, int page) {
#pragma unroll
                    for (int h = 0; h < L::HALVES; ++h)
                        tma_cache(dst + uint32_t(h * L::HALF + row * 128), map, 64 * h, g, slot_in, page, &full[s]);
                });
            }
        }
        report_bad(bad, status);
        if (!v && plan.q_copies && ok) {  // the run is over
            if (qi > 0) ok = __all_sync(0xffffffffu, wait_phase(&ctl->q_free, (qi - 1) & 1, abort_flag, wait_ns, status));
            if (ok && elect_one()) {
                *reinterpret_cast<volatile int *>(&ctl->item) = 0;
                mbar_arrive(&ctl->q_ready);
            }
            __syncwarp();
        }
        // every copy issued must land before the CTA exits
        if (lane == 0) {
            for (int j = max(0, blocks - 2); j < blocks; ++j)
                mbar_wait_bounded(&full[j & 1], (j >> 1) & 1, drain_ns(wait_ns), status);
            if (!v && plan.q_copies && qi > 0 && !ok) mbar_wait_bounded(&ctl->q_ready, (qi - 1) & 1, drain_ns(wait_ns), status);
        }
        __syncwarp();
    } else if (warp == W_MMA || warp == W_MMA + 1) {
        // ---- MMAs of lane w, by one thread
        const int w = warp - W_MMA;
        constexpr uint32_t type = is_half<T> ? 0u : (1u << 7) | (1u << 10);
        const int nd = uniform((a.dim + 15) / 16);  // 16-feature steps that hold anything
        const uint32_t idesc_s = (1u << 4) | type | (uint32_t(kStep >> 3) << 17) | (uint32_t(kRows >> 4) << 24);
        const uint32_t idesc_o = (1u << 4) | type | (1u << 16) | (uint32_t(nd * 2) << 17) | (uint32_t(kRows >> 4) << 24);
        auto wait_on = [&](uint64_t *bar, uint32_t parity) { return wait_phase(bar, parity, abort_flag, wait_ns, status); };
        // uniform values and an elected lane: with values that the compiler takes for divergent, an MMA's issue took 100
        // cycles instead of the 48 (N = 64) or 64 that it runs for; offsets never carry out of a descriptor's address field
        const uint64_t dk[2] = {desc_k(sK), desc_k(sK + L::TILE)};
        const uint64_t dv[2] = {desc_mn(sV, L::HALF), desc_mn(sV + L::TILE, L::HALF)};
        const uint32_t t_s = tmem + uint32_t(w * 128), t_o = tmem + kOCol + uint32_t(w * 128);
        // the MMAs of one item by this lane
        auto issue_item = [&](auto both, int steps, uint64_t dq, int done) -> bool {
            constexpr bool TWO = decltype(both)::value;
            const int from = blocks + (TWO ? 0 : w);
            bool ok = true;
            auto issue_s = [&](int u) -> bool {
                const int j = from + (TWO ? u >> 1 : u & ~1), h = u & 1;
                if (!h && !wait_on(&ctl->k_full[j & 1], (j >> 1) & 1)) return false;
                tc_fence_after();
                const uint64_t db = ((j & 1) ? dk[1] : dk[0]) + uint64_t(h * (kStep * 128 >> 4));
#pragma unroll
                for (int kk = 0; kk < DP / 16; ++kk) {
                    const uint64_t off = uint64_t((((kk >> 2) * L::HALF) >> 4) + 2 * (kk & 3));
                    if (kk < nd) tc_mma_f16(t_s + uint32_t(h * 64), dq + off, db + off, idesc_s, kk > 0);
                }
                tc_commit(&ctl->s_full[w][h]);
                if (h) {
                    tc_commit(&ctl->k_empty[j & 1]);
                    if (!TWO) tc_commit(&ctl->k_empty[j & 1]);
                }
                if (u == steps - 1) tc_commit(&ctl->q_free);
                return true;
            };
            for (int u = 0; u < 2 && u < steps && ok; ++u) ok = issue_s(u);
            for (int u = 0; u < steps && ok; ++u) {
                const int j = from + (TWO ? u >> 1 : u & ~1), h = u & 1;
                // (P first: its groups have then seen the whole item before end, so that V's parity, whose slot the other
                // lane may have used last, is read no earlier than one phase before)
                ok = wait_on(&ctl->p_full[w][h], ((done + u) >> 1) & 1) && (h || wait_on(&ctl->v_ready[j & 1], (j >> 1) & 1));
                if (!ok) break;
                tc_fence_after();
                const uint64_t db = ((j & 1) ? dv[1] : dv[0]) + uint64_t(h * (kStep * 128 >> 4));
                const uint32_t p = t_s + uint32_t(h * 64);
#pragma unroll
                for (int kk = 0; kk < kStep / 16; ++kk) {
                    const uint64_t bk = db + uint64_t(kk * 2048 >> 4);
                    mma_ts(t_o, p + uint32_t(kk * 8), bk, idesc_o, kk > 0 ? 1u : uint32_t(u > 0));
                    if constexpr (SPLIT_P) mma_ts(t_o, p + uint32_t(32 + kk * 8), bk, idesc_o, 1u);
                }
                tc_commit(&ctl->o_done[w]);
                if (u == steps - 1) tc_commit(&ctl->item_done[w]);
                if (h) {
                    tc_commit(&ctl->v_empty[j & 1]);
                    if (!TWO) tc_commit(&ctl->v_empty[j & 1]);
                }
                if (u + 2 < steps) ok = issue_s(u + 2);
            }
            return ok;
        };
        // Items come with Q (nb blocks, one or two tiles), so that nothing but MMAs and waits stands here; the warp takes them,
        // one lane issues.
        int done = 0;  // this lane's steps before the item
        for (;; ++qi) {
            bool ok = __all_sync(0xffffffffu, wait_on(&ctl->q_ready, qi & 1));
            const int item = ok ? uniform(*reinterpret_cast<volatile int *>(&ctl->item)) : 0, nb = item >> 1;
            if (nb == 0) break;
            const bool two = item & 1;
            const int steps = two ? 2 * nb : 2 * ((nb + 1 - w) >> 1);
            const uint64_t dq = desc_k(sQ + uint32_t(two ? w * L::TILE : 0));
            if (elect_one()) {
                if (steps == 0) tc_commit(&ctl->q_free);
                ok = two ? issue_item(bool_c<true>{}, steps, dq, done) : issue_item(bool_c<false>{}, steps, dq, done);
            }
            __syncwarp();
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            blocks = uniform(blocks + nb);
            done = uniform(done + steps);
        }
        if (elect_one()) tc_commit(&ctl->drain);  // when all of this lane's MMAs have ended
        __syncwarp();
    } else if (warp == W_SOFT - 1) {
        // ---- V: slots that some row of the item must not multiply
        bool ok = true;
        for (; ok && walk.more(); next_item(ok)) {
            if (walk.nb == 0) continue;
            ++qi;
            const RowSpan rs = walk.it.see;
            const int first = walk.first, last = walk.last;
            for (int j = 0; j < walk.nb; ++j, ++blocks) {
                const int slot = blocks & 1;
                ok = __all_sync(0xffffffffu, wait_phase(&ctl->v_full[slot], (blocks >> 1) & 1, abort_flag, wait_ns, status));
                if (!ok) break;
                const int key0 = (walk.block0 + j) * kBlock;
                // rows [0, r0) and [r1, 128) of the block
                const int r0 = min(kBlock, max(0, max(first, rs.lo_all) - key0)), r1 = max(r0, min(kBlock, min(last, rs.hi_all) - key0));
                if (r0 > 0 || r1 < kBlock) {
                    uint8_t *v = smem + L::OFF_V + slot * L::TILE;
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
                                ctl->poisoned[qi & 3] = qi;  // (read behind the MMAs that follow v_ready)
                            }
                        }
                    }
                    fence_proxy_async_smem();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl->v_ready[slot]);
            }
        }
    } else if (warp == W_CLAIM) {
        // ---- claims whole items, one at a time: CTAs of this grid that have not started are taken over, so that the next
        // item's copies run under this one's end
        if constexpr (!SPLIT) if (walk.left > 0) {
            ItemFinder finder(a);
            uint32_t asked = 0;
            for (;; ++claims) {
                const int slot = claims & 1;
                // (blocks are copied meanwhile, the last of the item before and this one's, each of which may take the limit)
                walk.more();
                const uint64_t limit = wait_ns >> 32 ? wait_ns : wait_ns * uint64_t(walk.nb + 8);
                bool ok = __all_sync(0xffffffffu, doze_phase(&ctl->want, claims & 1, abort_flag, limit, status));
                if (ok && claims >= 2)
                    ok = __all_sync(0xffffffffu, wait_phase(&ctl->item_free[slot], ((claims >> 1) - 1) & 1, abort_flag, wait_ns, status));
                if (!ok) break;
                Item it = {};
                for (int index = 0; index >= 0 && it.left == 0; ++asked) {  // (indices past the last item have none)
                    if (lane == 0) {
                        mbar_expect_tx(&ctl->answered, 16);
                        request_cta(&ctl->answer, &ctl->answered);
                    }
                    __syncwarp();
                    ok = __all_sync(0xffffffffu, wait_phase(&ctl->answered, asked & 1, abort_flag, wait_ns, status));
                    if (!ok) break;
                    index = uniform(requested_cta(&ctl->answer));
                    fence_proxy_async_smem();  // (read before the next answer is written)
                    __syncwarp();
                    if (index >= 0) it = finder.find(index, status);
                }
                if (!ok) {  // the answer must not come after the CTA has left
                    if (lane == 0) mbar_wait_bounded(&ctl->answered, asked & 1, drain_ns(wait_ns), status);
                    __syncwarp();
                    break;
                }
                if (lane == 0) {
                    ctl->next[slot] = it;
                    mbar_arrive(&ctl->item_full[slot]);
                }
                __syncwarp();
                if (it.left == 0) break;
                walk.begin(&it);
            }
        }
    } else {
        // ---- softmax groups.  After a wait that was given up a warp walks on without waiting or computing, so that every
        // warp meets every barrier.
        const int w = (warp - W_SOFT) >> 2;
        const uint32_t tl = uint32_t((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + tl + uint32_t(w * 128), to = tmem + tl + kOCol + uint32_t(w * 128);
        const int r = (warp & 3) * 32 + lane;                        // row in the tile = TMEM lane
        uint8_t *const stage = smem + L::OFF_STAGE + (warp - W_SOFT) * 4096;
        // scores stay unscaled; scale2 > 0 enters with the exponential (a zero scale as a tiny one, so that -inf stays)
        const float scale2 = fmaxf(fabsf(a.scale) * 1.4426950408889634f, 1e-30f);
        const uint64_t scale22 = pair(scale2, scale2);
        uint32_t phase = 0;  // bit 0: this lane's pairs of steps before the item (they are even), bit 1: its items with steps, modulo 2
        bool ok = true;
        // one warp's wait decides for both groups whether there is a next item: all of them meet the same barriers
        auto next_of_groups = [&]() {
            if constexpr (SPLIT) {
                walk.next();
            } else {
                const int slot = claims & 1;
                if (warp == W_SOFT) {
                    const bool got = __all_sync(0xffffffffu, wait_phase(&ctl->item_full[slot], (claims >> 1) & 1, abort_flag, wait_ns, status));
                    if (lane == 0) ctl->soft_go[slot] = got;
                    __syncwarp();
                }
                groups_sync();
                if (claims > 0 && lane == 0) mbar_arrive(&ctl->item_free[slot ^ 1]);  // (the one before is done with)
                if (*reinterpret_cast<volatile int *>(&ctl->soft_go[slot])) ++claims;
                else claims = -1;
            }
        };
        for (;; next_of_groups()) {
        if constexpr (!SPLIT) {
            if (claims < 0) {
                ok = false;
                break;
            }
            walk.begin(&ctl->next[claims == 0 ? 2 : (claims - 1) & 1]);
        }
        if (!walk.more()) break;
        if (walk.skip()) continue;
        const SeqSpan sp = walk.sp;
        const RowSpan rs = walk.it.see;
        const int b = walk.b, g = walk.g, row0 = walk.row0, rows = walk.rows, nt = walk.nt, nb = walk.nb, steps = walk.steps(w);
        const int first = walk.first, last = walk.last;
        const int row = (nt == 2 ? w * kRows : 0) + r;               // row of the item
        const KeyRange kr = row < rows ? keys_of(sp, (row0 + row) / G, a.window, a.causal) : KeyRange{0, INT32_MAX};  // (rows past the end: never written)
        const int lo = max(kr.lo, first), hi = min(kr.hi, last);
        if (nb > 0 && !plan.q_copies) {
            // both groups bring the rows of Q into the swizzled tiles, once no S of the item before reads them
            if (ok && qi > 0) ok = __all_sync(0xffffffffu, wait_phase(&ctl->q_free, (qi - 1) & 1, abort_flag, wait_ns, status));
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
                    const int rr = r_first + k * STEP;
                    *reinterpret_cast<uint4 *>(smem + (nt == 2 ? w * L::TILE : 0) + (c >> 3) * L::HALF + rr * 128 +
                                               (((c & 7) ^ (rr & 7)) << 4)) =
                        make_uint4(x[k].x ^ flip, x[k].y ^ flip, x[k].z ^ flip, x[k].w ^ flip);
                }
            fence_proxy_async_smem();
            groups_sync();
            if (ok && threadIdx.x == 32 * W_SOFT) {
                *reinterpret_cast<volatile int *>(&ctl->item) = 2 * nb + (nt == 2);
                mbar_arrive(&ctl->q_ready);
            }
        }
        if (nb > 0) ++qi;
        float m = -INFINITY, l = 0.f;
        for (int u = 0; u < steps && ok; ++u) {
            ok = __all_sync(0xffffffffu, wait_phase(&ctl->s_full[w][u & 1], (phase ^ uint32_t(u >> 1)) & 1, abort_flag, wait_ns, status));
            if (!ok) break;
            tc_fence_after();
            const int key0 = (walk.block0 + walk.block(w, u)) * kBlock + (u & 1) * kStep;
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
            const float neg = mu == -INFINITY ? 0.f : fmaf(-mu, scale2, weight_lift<T>);
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
        if (ok && steps > 0) {
            // (a barrier of its own: P V of the last two steps may both have ended by now, and a parity tells a phase only
            // from its neighbours)
            ok = __all_sync(0xffffffffu, wait_phase(&ctl->item_done[w], phase >> 1, abort_flag, wait_ns, status));
            phase ^= 2;
            tc_fence_after();
        }
        phase ^= uint32_t(steps >> 1) & 1;
        // one tile: the groups hold the softmax of the even and odd blocks of the same rows (and tensor-memory lanes);
        // each learns the other's m and l, and they take the output's pieces in turn
        float scale_own = 1.f, scale_other = 0.f;
        if (nt == 1) {
            float2 *mine = reinterpret_cast<float2 *>(stage);
            const float2 *other = reinterpret_cast<const float2 *>(smem + L::OFF_STAGE + (((warp - W_SOFT) + 4) & 7) * 4096);
            tc_fence_before();
            mine[lane] = make_float2(m, l);
            groups_sync();
            tc_fence_after();
            const float2 x = other[lane];
            groups_sync();
            const float top = fmaxf(m, x.x);  // (m == top holds where both are -inf)
            scale_own = m == top ? 1.f : fast_ex2((m - top) * scale2);
            scale_other = x.x == top ? 1.f : fast_ex2((x.x - top) * scale2);
            l = l * scale_own + x.y * scale_other;
            m = top;
        }
        const bool has_own = steps > 0, has_other = nt == 1 && walk.steps(1 - w) > 0;
        const uint32_t to_other = tmem + tl + kOCol + uint32_t((1 - w) * 128);
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
                if (p < 0) continue;  // (read as zeros)
                const T *v = static_cast<const T *>(a.v) + p * a.page_stride +
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
        if (ok) {
            const bool mine = row < rows, whole = walk.whole();
            const float inv = whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;  // no key: zeros
            const int64_t part = int64_t(walk.slot()) * kCtaRows;
            if (!whole) {
                if (mine && (nt == 2 || w == 0)) part_ml[part + row] = make_float2(m == -INFINITY ? m : m * scale2, l);
                if (threadIdx.x == 32 * W_SOFT)
                    pieces[walk.slot()] = make_int4(b + 1, row0, g, walk.u + walk.take == walk.units);
            }
            const bool poisoned = nb > 0 && *reinterpret_cast<volatile int *>(&ctl->poisoned[qi & 3]) == qi;
            // Rows leave through shared memory, 128 bytes of each at a time, so that eight lanes store one row's piece.
            auto put = [&](auto *to_rows, int64_t t_stride, int64_t h_stride, bool partial) {
                using E = typename std::remove_pointer<decltype(to_rows)>::type;
                constexpr int W = 128 / sizeof(E);  // columns of a piece: 32 in f32, 64 in 16 bits
                int64_t at[8];                      // where the rows that this lane stores a part of go
                const int r_out = row - lane + (lane >> 3);
                int i = (row0 + r_out) / G, hh = (row0 + r_out) % G;
                const int i_step = 4 / G, h_step = 4 % G;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    at[k] = partial ? (part + r_out + 4 * k) * a.dim : (int64_t(sp.q0) + i) * t_stride + int64_t(g * G + hh) * h_stride;
                    i += i_step;
                    hh += h_step;
                    if (hh >= G) {
                        hh -= G;
                        ++i;
                    }
                }
                for (int c0 = nt == 1 ? w * W : 0; c0 < a.dim; c0 += nt == 1 ? 2 * W : W) {
#pragma unroll
                    for (int half = 0; half < W / 32; ++half) {
                        const int c = c0 / 32 + half;
                        uint32_t o[32];
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = 0u;
                        if (has_own) {
                            tm_ld32(to + uint32_t(c * 32), o);
                            tm_wait_ld(o);
                        }
                        if (has_other) {
                            uint32_t x[32];
                            tm_ld32(to_other + uint32_t(c * 32), x);
                            tm_wait_ld(x);
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                o[e] = __float_as_uint((has_own ? __uint_as_float(o[e]) * scale_own : 0.f) + __uint_as_float(x[e]) * scale_other);
                        }
                        if (poisoned && mine) add_hidden(c, o);
#pragma unroll
                        for (int e0 = 0; e0 < 32; e0 += 16 / int(sizeof(E))) {
                            uint4 v;
                            auto f = [&](int e) { return __uint_as_float(o[e0 + e]) * inv; };
                            if constexpr (sizeof(E) == 4)
                                v = make_uint4(__float_as_uint(f(0)), __float_as_uint(f(1)), __float_as_uint(f(2)), __float_as_uint(f(3)));
                            else
                                v = make_uint4(pack16<E>(f(0), f(1)), pack16<E>(f(2), f(3)), pack16<E>(f(4), f(5)), pack16<E>(f(6), f(7)));
                            const int piece = (half * 32 + e0) * int(sizeof(E)) / 16;
                            *reinterpret_cast<uint4 *>(stage + lane * 128 + ((piece ^ (lane & 7)) << 4)) = v;
                        }
                    }
                    __syncwarp();
                    const int piece = lane & 7, col = c0 + piece * (16 / int(sizeof(E)));
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const int rr = k * 4 + (lane >> 3);
                        const uint4 v = *reinterpret_cast<const uint4 *>(stage + rr * 128 + ((piece ^ (rr & 7)) << 4));
                        if (r_out + 4 * k < rows && col < a.dim) *reinterpret_cast<uint4 *>(to_rows + at[k] + col) = v;
                    }
                    __syncwarp();
                }
            };
            if (whole) put(static_cast<TO *>(a.out), a.out_token, a.out_head, false);
            else put(part_o, 0, 0, true);
        }
        // the next item's first P V writes over O: not before this group (one tile: both groups) has read it
        tc_fence_before();
        if (nt == 1 && SPLIT) groups_sync();  // (whole items: they meet before the next one)
        }
        if (!plan.q_copies && warp == W_SOFT && ok) {  // the run is over
            if (qi > 0) ok = __all_sync(0xffffffffu, wait_phase(&ctl->q_free, (qi - 1) & 1, abort_flag, wait_ns, status));
            if (ok && lane == 0) {
                *reinterpret_cast<volatile int *>(&ctl->item) = 0;
                mbar_arrive(&ctl->q_ready);
            }
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

// Joins the pieces of the item that run `blockIdx.x` begins and does not end: its own last
// one, and the first ones of the runs after it up to the one that ends it, in that
// order.  A warp takes four rows, with two pieces of each in flight.
template <typename TO>
__global__ void __launch_bounds__(32 * kJoinWarps, 6)
chunk_join_kernel(const PagedArgs a, const float *__restrict__ part_o, const float2 *__restrict__ part_ml,
                  const Piece *__restrict__ pieces, int ctas) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int c0 = blockIdx.x, G = a.heads / a.kv_heads, lane = threadIdx.x & 31;
    const Piece p = pieces[2 * c0 + 1];
    if (p.x == 0) return;
    int c1 = ctas;  // the run that ends the item
    for (int c = c0 + 1; c < ctas; c += 32) {
        const unsigned ends = __ballot_sync(0xffffffffu, c + lane < ctas && pieces[2 * (c + lane)].w != 0);
        if (ends) {
            c1 = c + __ffs(ends) - 1;
            break;
        }
    }
    if (c1 == ctas) return;
    const int b = p.x - 1, row0 = p.y, g = p.z, count = c1 - c0 + 1;
    bool ignore = false;
    const SeqSpan sp = seq_span(a.batch, b, ignore);  // (reported by the launch before)
    const int rows = min(kCtaRows, int(int64_t(sp.n) * G - row0));
    const int r0 = (blockIdx.y * kJoinWarps + (threadIdx.x >> 5)) * kJoinRows;
    if (r0 >= rows) return;
    const bool mine = 4 * lane < a.dim;
    float m[kJoinRows], l[kJoinRows];
    float4 o[kJoinRows];
#pragma unroll
    for (int r = 0; r < kJoinRows; ++r) {
        m[r] = -INFINITY;
        l[r] = 0.f;
        o[r] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    constexpr int AHEAD = 2;
    for (int k0 = 0; k0 < count; k0 += AHEAD) {
        float2 ml[AHEAD][kJoinRows];
        float4 x[AHEAD][kJoinRows];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k)
#pragma unroll
            for (int r = 0; r < kJoinRows; ++r) {
                ml[k][r] = make_float2(-INFINITY, 0.f);
                x[k][r] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (k0 + k < count && r0 + r < rows) {
                    const int64_t at = int64_t(k0 + k == 0 ? 2 * c0 + 1 : 2 * (c0 + k0 + k)) * kCtaRows + r0 + r;
                    ml[k][r] = part_ml[at];
                    if (mine) x[k][r] = *reinterpret_cast<const float4 *>(part_o + at * a.dim + 4 * lane);
                }
            }
#pragma unroll
        for (int r = 0; r < kJoinRows; ++r) {
            float next = m[r];
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) next = fmaxf(next, ml[k][r].x);
            const float keep = m[r] == next ? 1.f : fast_ex2(m[r] - next);
            l[r] *= keep;
            o[r].x *= keep;
            o[r].y *= keep;
            o[r].z *= keep;
            o[r].w *= keep;
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) {
                const float f = ml[k][r].x == next ? 1.f : fast_ex2(ml[k][r].x - next);
                l[r] = fmaf(f, ml[k][r].y, l[r]);
                o[r].x = fmaf(f, x[k][r].x, o[r].x);
                o[r].y = fmaf(f, x[k][r].y, o[r].y);
                o[r].z = fmaf(f, x[k][r].z, o[r].z);
                o[r].w = fmaf(f, x[k][r].w, o[r].w);
            }
            m[r] = next;
        }
    }
#pragma unroll
    for (int r = 0; r < kJoinRows; ++r)
        if (mine && r0 + r < rows) {
            const int i = (row0 + r0 + r) / G, h = g * G + (row0 + r0 + r) % G;
            const float inv = l[r] == 0.f ? 0.f : 1.f / l[r];
            store4(static_cast<TO *>(a.out) + (int64_t(sp.q0) + i) * a.out_token + int64_t(h) * a.out_head + 4 * lane, o[r].x * inv,
                   o[r].y * inv, o[r].z * inv, o[r].w * inv);
        }
}

struct ChunkLaunch {
    ChunkPlan plan;
    int ctas;
};

// tiles: at most, each sequence leaves less than one unfilled
int64_t tile_bound(int64_t group, int64_t seqs, int64_t tokens) {
    return (tokens * group + std::min(seqs, tokens) * (kCtaRows - 1)) / kCtaRows;
}

// Items are cut where one CTA an item would leave the SMs idle for longer than cutting
// costs: with fewer than two turns of items, the last turn's idle share times an item's
// blocks (1.7 us each), against about 14 us for the partial results and the join.  Measured:
// 512 tokens over 32768 keys, 8 key heads (64 items of 256 blocks) 207 us cut (195 since)
// and 229 in chunks of keys; 1216 tokens over 8192 (152 items) 131 cut, 101 whole (97 since); 1024 of a
// prompt (128 items of up to 8 blocks) 34 cut, 23 whole.
ChunkLaunch chunk_launch(int64_t items, int64_t max_q, int64_t span) {
    ChunkLaunch r = {};
    const int64_t blocks = std::max<int64_t>(1, (span - std::min(max_q, span) / 2) / kBlock);
    const int64_t idle = (items + kNumSms - 1) / kNumSms * kNumSms - items;
    r.plan.split = items < 2 * kNumSms && idle * blocks > 8 * kNumSms;
    const int64_t units = items * (kStartUnits + span / kBlock + 2);
    r.ctas = int(r.plan.split ? std::min<int64_t>(kNumSms, (units + kMinUnits - 1) / kMinUnits) : items);
    return r;
}

size_t chunk_ws_bytes(int64_t ctas, int64_t dim) {
    return size_t(2 * ctas * kCtaRows) * size_t(dim * 4 + 8) + size_t(2 * ctas) * sizeof(Piece);
}

// Tensor map of q whose boxes are a 128-row tile's 64 features: G heads of 128 / G tokens.
template <typename T>
cudaError_t q_map(const PagedArgs &a, CUtensorMap *map) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return cudaErrorNotSupported;
    const int G = a.heads / a.kv_heads;
    const cuuint64_t dims[3] = {cuuint64_t(a.dim), cuuint64_t(a.heads), cuuint64_t(a.batch.tokens)};
    auto bytes = [&](int64_t s) { return cuuint64_t(s ? s : a.dim) * 2; };  // (0: an axis of one element)
    const cuuint64_t strides[2] = {bytes(a.q_head), bytes(a.q_token)};
    const cuuint32_t box[3] = {64, cuuint32_t(G), cuuint32_t(kRows / G)}, step[3] = {1, 1, 1};
    if (enc(map, is_half<T> ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(a.q), dims,
            strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    return cudaSuccess;
}

template <typename T, typename TO, int DP>
cudaError_t launch_chunk(const PagedArgs &a, void *ws, const LaunchCtx &ctx) {
    using L = ChunkLayout<DP>;
    const int64_t G = a.heads / a.kv_heads, items = tile_bound(G, a.batch.seqs, a.batch.tokens) * a.kv_heads;
    const int64_t span = key_span(a.batch.max_q, a.batch.max_kv, a.window);
    if (items > INT32_MAX / (span / kBlock + 8)) return cudaErrorInvalidValue;
    ChunkLaunch r = chunk_launch(items, a.batch.max_q, span);
    r.plan.box_rows = std::min(a.batch.page_size & -a.batch.page_size, kBlock);
    // a stride of 0 along more than one head or token (a broadcast q) has no tensor map
    r.plan.q_copies = kRows % G == 0 && a.scale >= 0.f && (a.q_head || a.heads == 1) && (a.q_token || a.batch.tokens == 1);
    CUtensorMap km, vm, qm = {};
    cudaError_t e = cache_maps<T>(a, r.plan.box_rows, &km, &vm);
    if (e == cudaSuccess && r.plan.q_copies) e = q_map<T>(a, &qm);
    if (e != cudaSuccess) return e;
    auto kernel = r.plan.split ? paged_chunk_kernel<T, TO, DP, true> : paged_chunk_kernel<T, TO, DP, false>;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::BYTES);
    if (e != cudaSuccess) return e;
    const int64_t slots = 2 * int64_t(r.ctas) * kCtaRows;
    float *po = r.plan.split ? static_cast<float *>(ws) : nullptr;
    float2 *pml = r.plan.split ? reinterpret_cast<float2 *>(po + slots * a.dim) : nullptr;
    Piece *pieces = r.plan.split ? reinterpret_cast<Piece *>(pml + slots) : nullptr;
    e = launch_dependent(kernel, dim3(unsigned(r.ctas)), kThreads, L::BYTES, ctx.stream, km, vm, qm, a, r.plan, po, pml, pieces,
                         ctx.status, ctx.wait_ns);
    if (e != cudaSuccess || !r.plan.split) return e;
    return launch_dependent(chunk_join_kernel<TO>, dim3(unsigned(r.ctas), kJoinParts), 32 * kJoinWarps, 0, ctx.stream, a,
                            static_cast<const float *>(po), static_cast<const float2 *>(pml), static_cast<const Piece *>(pieces), r.ctas);
}

template <typename T, typename TO>
cudaError_t launch_chunk_io(const PagedArgs &a, void *ws, const LaunchCtx &ctx) {
    return a.dim <= 64 ? launch_chunk<T, TO, 64>(a, ws, ctx) : launch_chunk<T, TO, 128>(a, ws, ctx);
}

}  // namespace

size_t attention_paged_chunk_ws_bytes(int64_t heads, int64_t kv_heads, int64_t dim, int64_t seqs, int64_t tokens, int64_t max_q,
                                      int64_t max_kv) {
    const ChunkLaunch r = chunk_launch(tile_bound(heads / kv_heads, seqs, tokens) * kv_heads, max_q, max_kv);  // (a window only shortens the span)
    return r.plan.split ? chunk_ws_bytes(r.ctas, dim) : 0;
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
