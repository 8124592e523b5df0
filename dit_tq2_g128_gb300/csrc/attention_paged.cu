// Attention of a step's new tokens over a paged key/value cache: few query rows.
//
// Mathematics.  The rows of one sequence that share a key head (its new tokens
// times the query heads of the group, R = n * G of them) read the same keys, so
// a CTA takes all of them at once: S^T = K Q^T, P = exp2(S log2(e) scale - m),
// O^T += V^T P^T over tiles of 64 keys, with the running maximum m and sum l of
// the softmax.  Keys are the rows (M) of both products and the query rows their
// columns (N = 8 to 32): decoding wastes no tensor rows as it would with the
// queries in M.
//
// Bound by memory: 2 R flops per byte of cache at 16 bits, below the warp-level
// tensor path's rate for few rows.  The tcgen05 path (attention_paged_chunk.cu) needs
// 128 rows in M and takes over above rows_max.
//
// Work is shared out evenly: the (sequence, key head) pairs' tiles, in one line, are
// cut into as many equal runs as there are CTAs (two an SM), wherever that falls; a
// pair that is cut leaves (m, l, O) of its pieces in the workspace and a second,
// dependent launch joins them in order.  So a batch of very different lengths keeps
// every SM busy to the end, and a CTA starts once.  (Cut into chunks of 1024 keys, 64
// sequences of 3000 keys, eight key heads of 128, took 135 us; shared out 123 us, 94 %
// of the copy rate.)
//
// A CTA has four consumer warps of 16 keys each a tile and one producer warp, which
// runs ahead through all of the CTA's pairs.  It looks pages up 32 boxes at a time and
// copies rows by tensor copies with the 128-byte swizzle into a ring of three tiles (96
// KB at 128 features; two CTAs an SM keep 192 KB in flight).  A copy's box is the
// largest power of two of rows that divides the page size, so a box never crosses a
// page, whatever the page size; features past dim are filled with zeros by the copy.
// Every warp keeps its own m, l and O; they meet at the end of a pair, in the ring's
// slot of its last tile.
//
// Slots that no row sees are never multiplied: their scores are replaced by
// -inf and their rows of V are zeroed in shared memory (0 * NaN is NaN).  Where
// some rows see a key and others do not, values of V that are not finite are
// taken out of the product and added to the rows that see them.
#include <algorithm>

#include <cuda_bf16.h>

#include "paged_attention.cuh"

namespace tq2 {
namespace {

constexpr int kKeys = 64;       // keys of a tile
constexpr int kStages = 3;
constexpr int kConsumers = 4;   // warps, 16 keys of a tile each
constexpr int kThreads = 32 * (kConsumers + 1);
constexpr int kCtas = 2 * kNumSms;
constexpr int kMinTiles = 4;    // units of a run, at least, where pairs may be cut
constexpr int kWholeKeys = 512; // up to so many keys a pair stays whole (a join costs more than a CTA saves)

// Query rows per (sequence, key head) that this kernel takes; more go to the tcgen05
// kernel.  The limit is where O and S of a warp's 16 keys no longer fit its registers (168
// a thread at two CTAs an SM): 32 rows of 64 features (2 to 5 words spilled), 16 of 128.  Measured, this kernel
// against that one: 28 rows of 64, 16 sequences of 1000 keys 13.7 / 16.2 us, 32 rows, 64
// of 2000 keys 90 / 100, 21 rows, 16 of 1000 11.5 / 16.2 (8 of 200 keys, 32 rows: 9.8 /
// 8.9); 40 rows of 64, spilled, 64 of 2000 keys 126 / 100; 16 rows of 128, 64 of 2000
// keys 100 / 123; 24 rows of 128, spilled, 153 / 123.
constexpr int64_t rows_max(int64_t dim) { return dim <= 64 ? 32 : 16; }

template <int DP, int NT>
struct RowLayout {
    static constexpr int HALVES = DP / 64;
    static constexpr int HALF = kKeys * 128;           // one swizzled sub-tile of 64 features
    static constexpr int PLANE = HALF * HALVES;        // K (or V) of a tile
    static constexpr int RING = kStages * 2 * PLANE;
    static constexpr int ROWS = 8 * NT;
    static constexpr int OPAD = DP + 4;                // f32 row of the warps' exchange
    static_assert(kConsumers * 8 * OPAD * 4 <= 2 * PLANE, "eight rows' exchange lies in a slot");
    static constexpr int OFF_CTL = RING;
    static constexpr int OFF_ML = OFF_CTL + 128;       // m, l per warp and row, twice (pairs in turn)
    static constexpr int OFF_POISON = OFF_ML + 4 * kConsumers * ROWS * 4;
    static constexpr int BYTES = OFF_POISON + ROWS * DP * 4 + 1024;
};

struct RowCtl {
    uint64_t full[kStages], empty[kStages];
    int abort, poisoned;
    int b, g, t, left;  // where this CTA's run begins: sequence, key head, unit; its units
};
static_assert(sizeof(RowCtl) <= 128, "control block");

__device__ __forceinline__ void consumer_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
static_assert(32 * kConsumers == 128, "consumer_sync");

template <typename T>
__device__ __forceinline__ void mma_16x8(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (is_half<T>)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// How a call is shared out: `rows` query rows a pair at most, the rows of a copy, and
// whether pairs may be cut.
struct RowPlan {
    int rows;
    int box_rows;
    int split;
};

// The run of this CTA (one warp): `left` units from unit t of (b, g) on.  Block 0 also
// leaves each sequence's first unit and the units of a run for the join.
__device__ __forceinline__ void find_run(const PagedArgs &a, const RowPlan &plan, RowCtl *ctl, int *__restrict__ starts,
                                         unsigned int *status) {
    const int lane = threadIdx.x & 31;
    auto units_of = [&](int b) {  // of one key head
        bool bad = false;
        const int n = b < a.batch.seqs ? tiles_of(seq_span(a.batch, b, bad), a.window, a.causal, kKeys, plan.split).units : 0;
        report_bad(bad, status);
        return n;
    };
    const int head = units_of(lane);
    int total = int(__reduce_add_sync(0xffffffffu, unsigned(head))) * a.kv_heads;
    for (int base = 32; base < a.batch.seqs; base += 32)
        total += int(__reduce_add_sync(0xffffffffu, unsigned(units_of(base + lane)))) * a.kv_heads;
    const int ctas = int(gridDim.x), least = plan.split ? kMinTiles : 1;
    const int share = max(least, (total + ctas - 1) / ctas);
    const bool write = blockIdx.x == 0 && starts != nullptr;
    const int64_t from = int64_t(blockIdx.x) * share;
    int before = 0;
    if (lane == 0) {
        ctl->left = from < total ? int(min(int64_t(share), total - from)) : 0;
        if (write) starts[a.batch.seqs] = share;
    }
    if (from >= total && !write) return;
    for (int base = 0; base < a.batch.seqs; base += 32) {
        const int b = base + lane;
        const int per = base == 0 ? head : units_of(b), units = per * a.kv_heads;
        int upto = units;  // inclusive over the lanes
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, upto, d);
            if (lane >= d) upto += x;
        }
        upto += before;
        if (write && b < a.batch.seqs) starts[b] = upto - units;
        if (units > 0 && from >= upto - units && from < upto) {
            const int at = int(from) - (upto - units);
            ctl->b = b;
            ctl->g = at / per;
            ctl->t = at % per;
        }
        before = __shfl_sync(0xffffffffu, upto, 31);
        if (!write && from < before) return;
    }
}

// A CTA's run, pair by pair: every role walks it by itself.
struct RowWalk {
    const PagedArgs &a;
    const RowPlan &plan;
    int b, g, t, left;
    SeqSpan sp;
    RowSpan rs;
    TileSpan ts;
    // the current pair's part
    int first, last, tile0, tiles, take;

    __device__ __forceinline__ RowWalk(const PagedArgs &args, const RowPlan &p, const RowCtl *ctl)
        : a(args), plan(p), b(uniform(ctl->b)), g(uniform(ctl->g)), t(uniform(ctl->t)), left(uniform(ctl->left)) {
        if (left > 0) load();
    }
    __device__ __forceinline__ void load() {
        bool ignore = false;
        const SeqSpan s = seq_span(a.batch, b, ignore);  // (reported by find_run)
        sp = SeqSpan{uniform(s.q0), uniform(s.n), uniform(s.kv)};
        if (sp.n == 0) return;
        rs = rows_see(sp, 0, sp.n - 1, a.window, a.causal);
        ts = tiles_of(sp, a.window, a.causal, kKeys, plan.split);
    }
    __device__ __forceinline__ bool more() {
        if (left <= 0) return false;
        take = min(left, ts.units - t);
        const bool cut = ts.units > 1;  // units are tiles
        tile0 = ts.tile0 + (cut ? t : 0);
        tiles = cut ? take : ts.tiles;
        first = max(rs.lo, tile0 * kKeys);
        last = min(rs.hi, (tile0 + tiles) * kKeys);
        return true;
    }
    __device__ __forceinline__ bool whole() const { return t == 0 && take == ts.units; }
    // where a cut pair's piece goes: a run's first piece, begun by the run before, or its last
    __device__ __forceinline__ int slot() const { return 2 * int(blockIdx.x) + (t == 0); }
    __device__ __forceinline__ void next() {
        left -= take;
        t += take;
        if (t < ts.units) return;
        t = 0;
        if (++g < a.kv_heads) return;
        g = 0;
        while (left > 0 && ++b < a.batch.seqs) {
            load();
            if (sp.n > 0) break;
        }
    }
};

// DP: features padded to 64 or 128; NT: query rows in eights; SPLIT_P: the weights
// enter the second product as two terms, of bf16 as three (f32 outputs).
template <typename T, typename TO, int DP, int NT>
__global__ void __launch_bounds__(kThreads, 2)
paged_rows_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                  const PagedArgs a, const RowPlan plan, float *__restrict__ part_o, float2 *__restrict__ part_ml,
                  int *__restrict__ starts, unsigned int *status, uint64_t wait_ns) {
    using L = RowLayout<DP, NT>;
    constexpr bool SPLIT_P = sizeof(TO) == 4, THIRD = SPLIT_P && !is_half<T>;  // (three terms of bf16's 8 bits)
    extern __shared__ uint8_t rows_raw[];
    const uint32_t raw = smem_u32(rows_raw), pad = (1024u - (raw & 1023u)) & 1023u, base = raw + pad;
    uint8_t *smem = rows_raw + pad;
    RowCtl *ctl = reinterpret_cast<RowCtl *>(smem + L::OFF_CTL);
    float *poison = reinterpret_cast<float *>(smem + L::OFF_POISON);
    const int warp = uniform(int(threadIdx.x >> 5)), lane = threadIdx.x & 31;
    const int G = a.heads / a.kv_heads;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&ctl->full[s], 1);
            mbar_init(&ctl->empty[s], kConsumers);
        }
        ctl->abort = 0;
        ctl->poisoned = 0;
        fence_mbarrier_init();
    }
    // the tables, q and the cache may be written by the kernel before this one
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (warp == 0) find_run(a, plan, ctl, starts, status);
    __syncthreads();
    RowWalk walk(a, plan, ctl);
    int ring = 0;  // tiles so far, over all pairs

    if (warp == kConsumers) {
        // ---- producer: ahead through the run, as far as the ring has room
        bool bad = false, ok = true;
        for (; ok && walk.more(); walk.next()) {
            BoxPages boxes(a, walk.b, walk.tile0 * kKeys, kKeys, plan.box_rows, walk.first, walk.last);
            const int tiles = uniform(walk.tiles), g = uniform(walk.g);
            ring = uniform(ring);
            for (int it = 0; it < tiles; ++it, ++ring) {
                const int s = ring % kStages, u = ring / kStages;
                boxes.seek(it);
                if (u > 0) ok = __all_sync(0xffffffffu, wait_phase(&ctl->empty[s], (u - 1) & 1, &ctl->abort, wait_ns, status));
                if (!ok) break;
                const uint32_t stage = base + uint32_t(s * 2 * L::PLANE);
                const BoxRange br = boxes.range(it);
                if (lane == 0) mbar_expect_tx(&ctl->full[s], uint32_t((br.hi - br.lo) * boxes.rows * 256 * L::HALVES));
                __syncwarp();
                boxes.each(it, br, bad, [&](int row, int slot, int page) {
#pragma unroll
                    for (int h = 0; h < L::HALVES; ++h) {
                        tma_cache(stage + uint32_t(h * L::HALF + row * 128), &kmap, 64 * h, g, slot, page, &ctl->full[s]);
                        tma_cache(stage + uint32_t(L::PLANE + h * L::HALF + row * 128), &vmap, 64 * h, g, slot, page, &ctl->full[s]);
                    }
                });
            }
        }
        report_bad(bad, status);
        // What was issued lands before the CTA ends, whoever gave up: with three tiles or fewer this warp has waited for
        // nothing, so a consumer's wait may have run out unseen here.  (Else the consumers wait for the same phases.)
        if (lane == 0)
            for (int t = max(0, ring - kStages); t < ring; ++t)
                mbar_wait_bounded(&ctl->full[t % kStages], (t / kStages) & 1, drain_ns(wait_ns), status);
        return;
    }

    // ---- consumers: 16 keys of every tile.  After a wait that was given up a warp walks on without waiting or
    // computing, so that every warp meets every barrier.
    bool ok = true;
    for (int pairs = 0; walk.more(); walk.next(), ++pairs) {
        const SeqSpan sp = walk.sp;
        const RowSpan rs = walk.rs;
        const int g = walk.g, R = sp.n * G, first = walk.first, last = walk.last, tiles = walk.tiles;
        if (sp.n > 1) {  // (one token's keys are seen by all its rows or by none)
            consumer_sync();  // the pair before has been written
            for (int i = threadIdx.x; i < L::ROWS * DP; i += 32 * kConsumers) poison[i] = 0.f;
            if (threadIdx.x == 0) ctl->poisoned = 0;
            consumer_sync();
        }
        float m[NT][2], l[NT][2], o[NT][DP / 16][4];
        uint32_t q[NT][DP / 16][2];
        int lo[NT][2], hi[NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int r = t * 8 + (lane >> 2);
            const T *qr = static_cast<const T *>(a.q) + (int64_t(sp.q0) + r / G) * a.q_token + int64_t(g * G + r % G) * a.q_head;
#pragma unroll
            for (int kk = 0; kk < DP / 16; ++kk)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int d = kk * 16 + e * 8 + 2 * (lane & 3);
                    q[t][kk][e] = r < R && d < a.dim ? *reinterpret_cast<const uint32_t *>(qr + d) : 0u;
                }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int n = t * 8 + 2 * (lane & 3) + c;
                const KeyRange kr = keys_of(sp, n / G, a.window, a.causal);
                lo[t][c] = n < R ? kr.lo : 0;
                hi[t][c] = n < R ? kr.hi : 0;
                m[t][c] = -INFINITY;
                l[t][c] = 0.f;
            }
#pragma unroll
            for (int j = 0; j < DP / 16; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[t][j][e] = 0.f;
        }
        const float scale2 = a.scale * 1.4426950408889634f;
        const int arow = lane & 15, brow = (lane & 7) + ((lane >> 4) & 1) * 8;
        for (int it = 0; it < tiles && ok; ++it, ++ring) {
            const int s = ring % kStages;
            ok = __all_sync(0xffffffffu, wait_phase(&ctl->full[s], (ring / kStages) & 1, &ctl->abort, wait_ns, status));
            if (!ok) break;
            const int key0 = (walk.tile0 + it) * kKeys + warp * 16;
            const uint32_t ks = base + uint32_t(s * 2 * L::PLANE + warp * 16 * 128), vs = ks + L::PLANE;
            if (key0 < last && key0 + 16 > first) {
                const bool clean = key0 >= rs.lo_all && key0 + 16 <= min(rs.hi_all, last) && key0 >= first;
                if (!clean) {
                    // rows of V that no query row sees (or that this chunk does not own) become zeros; where only
                    // some see them, values that are not finite go to those rows' sums apart
                    uint8_t *vrow = smem + (vs - base) + (lane >> 1) * 128;
                    const int key = key0 + (lane >> 1);
                    const bool mine = key >= first && key < last;
                    for (int c = lane & 1; c < L::HALVES * 8; c += 2) {
                        uint4 *p = reinterpret_cast<uint4 *>(vrow + (c >> 3) * L::HALF + (((c & 7) ^ ((lane >> 1) & 7)) << 4));
                        if (!mine) {
                            *p = make_uint4(0, 0, 0, 0);
                        } else if (key < rs.lo_all || key >= rs.hi_all) {
                            uint4 w = *p;
                            if (any_nonfinite<T>(w)) {
                                take_nonfinite<T>(w, [&](int e, float x) {
                                    for (int n = 0; n < R; ++n) {
                                        const KeyRange kr = keys_of(sp, n / G, a.window, a.causal);
                                        if (key >= kr.lo && key < kr.hi) atomicAdd(&poison[n * DP + c * 8 + e], x);
                                    }
                                });
                                *p = w;
                                ctl->poisoned = 1;
                            }
                        }
                    }
                    __syncwarp();
                }
                // S^T = K Q^T, [16 keys] x [8 NT rows]
                float sc[NT][4], sd[NT][4];  // (two sums, of the even and odd steps: half the chain of dependent MMAs)
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sc[t][e] = sd[t][e] = 0.f;
#pragma unroll
                for (int kk = 0; kk < DP / 16; ++kk) {
                    uint32_t ka[4];
                    const int c = 2 * (kk & 3) + (lane >> 4);
                    ldsm4(ka, ks + uint32_t((kk >> 2) * L::HALF + arow * 128 + ((c ^ (arow & 7)) << 4)));
#pragma unroll
                    for (int t = 0; t < NT; ++t) mma_16x8<T>(kk & 1 ? sd[t] : sc[t], ka, q[t][kk][0], q[t][kk][1]);
                }
                uint32_t ph[NT][2], pl[NT][2], pt[NT][2];
#pragma unroll
                for (int t = 0; t < NT; ++t) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        sc[t][e] = (sc[t][e] + sd[t][e]) * scale2;
                        if (!clean) {
                            const int key = key0 + (lane >> 2) + (e >> 1) * 8, c = e & 1;
                            if (key < max(lo[t][c], first) || key >= min(hi[t][c], last)) sc[t][e] = -INFINITY;
                        }
                    }
                    // lazy rescale: m follows the maximum only when it grows by more than 2^8
                    const float x0 = fmaxf(sc[t][0], sc[t][2]), x1 = fmaxf(sc[t][1], sc[t][3]);
                    if (__any_sync(0xffffffffu, x0 > m[t][0] + 8.f || x1 > m[t][1] + 8.f)) {
                        float y0 = fmaxf(x0, m[t][0]), y1 = fmaxf(x1, m[t][1]);
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1) {
                            y0 = fmaxf(y0, __shfl_xor_sync(0xffffffffu, y0, d));
                            y1 = fmaxf(y1, __shfl_xor_sync(0xffffffffu, y1, d));
                        }
                        const float f0 = y0 == m[t][0] ? 1.f : fast_ex2(m[t][0] - y0);
                        const float f1 = y1 == m[t][1] ? 1.f : fast_ex2(m[t][1] - y1);
                        m[t][0] = y0;
                        m[t][1] = y1;
                        l[t][0] *= f0;
                        l[t][1] *= f1;
#pragma unroll
                        for (int j = 0; j < DP / 16; ++j) {
                            o[t][j][0] *= f0;
                            o[t][j][1] *= f1;
                            o[t][j][2] *= f0;
                            o[t][j][3] *= f1;
                        }
                    }
                    const float u0 = m[t][0] == -INFINITY ? 0.f : m[t][0] - weight_lift<T>;
                    const float u1 = m[t][1] == -INFINITY ? 0.f : m[t][1] - weight_lift<T>;
                    float p[4];
                    p[0] = fast_ex2(sc[t][0] - u0);
                    p[1] = fast_ex2(sc[t][1] - u1);
                    p[2] = fast_ex2(sc[t][2] - u0);
                    p[3] = fast_ex2(sc[t][3] - u1);
                    l[t][0] += p[0] + p[2];
                    l[t][1] += p[1] + p[3];
                    // the weights in the cache's type (the second product's operands have one type); an f32 output
                    // keeps their remainder as a second term, and in bf16 a third
                    const uint32_t w0 = pack16<T>(p[0], p[1]), w1 = pack16<T>(p[2], p[3]);
                    ph[t][0] = transpose_8x8(w0);
                    ph[t][1] = transpose_8x8(w1);
                    if constexpr (SPLIT_P) {
                        float h[4];
                        unpack16<T>(w0, h[0], h[1]);
                        unpack16<T>(w1, h[2], h[3]);
                        const uint32_t l0 = pack16<T>(p[0] - h[0], p[1] - h[1]), l1 = pack16<T>(p[2] - h[2], p[3] - h[3]);
                        pl[t][0] = transpose_8x8(l0);
                        pl[t][1] = transpose_8x8(l1);
                        if constexpr (THIRD) {
                            float x[4];
                            unpack16<T>(l0, x[0], x[1]);
                            unpack16<T>(l1, x[2], x[3]);
                            pt[t][0] = transpose_8x8(pack16<T>(p[0] - h[0] - x[0], p[1] - h[1] - x[1]));
                            pt[t][1] = transpose_8x8(pack16<T>(p[2] - h[2] - x[2], p[3] - h[3] - x[3]));
                        }
                    }
                }
                // O^T += V^T P^T
#pragma unroll
                for (int j = 0; j < DP / 16; ++j) {
                    uint32_t va[4];
                    const int c = 2 * (j & 3) + ((lane >> 3) & 1);
                    ldsm4_t(va, vs + uint32_t((j >> 2) * L::HALF + brow * 128 + ((c ^ (brow & 7)) << 4)));
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        mma_16x8<T>(o[t][j], va, ph[t][0], ph[t][1]);
                        if constexpr (SPLIT_P) mma_16x8<T>(o[t][j], va, pl[t][0], pl[t][1]);
                        if constexpr (THIRD) mma_16x8<T>(o[t][j], va, pt[t][0], pt[t][1]);
                    }
                }
                if (!clean) fence_proxy_async_smem();  // this warp wrote where the next copies land
            }
            __syncwarp();
            if (it + 1 < tiles && lane == 0) mbar_arrive(&ctl->empty[s]);  // the last tile's slot is kept for the exchange
        }
        // m and l of this warp's keys
        float *wm = reinterpret_cast<float *>(smem + L::OFF_ML) + (pairs & 1) * 2 * kConsumers * L::ROWS;
        float *wl = wm + kConsumers * L::ROWS;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float x = l[t][c];
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
                if (lane < 4) {
                    wm[warp * L::ROWS + t * 8 + 2 * lane + c] = m[t][c];
                    wl[warp * L::ROWS + t * 8 + 2 * lane + c] = x;
                }
            }
        const int kept = tiles > 0 ? (ring + kStages - 1) % kStages : 0;  // slot of the last tile
        float *ob = reinterpret_cast<float *>(smem + kept * 2 * L::PLANE);  // [warp][8 rows][OPAD]
        const bool whole = walk.whole();
#pragma unroll
        for (int t = 0; t < NT; ++t) {  // eight rows at a time
            consumer_sync();
#pragma unroll
            for (int c = 0; c < 2 && tiles > 0; ++c) {  // (a pair without keys has no slot, and zeros)
                const int n = 2 * (lane & 3) + c;
                float top = wm[t * 8 + n];
#pragma unroll
                for (int w = 1; w < kConsumers; ++w) top = fmaxf(top, wm[w * L::ROWS + t * 8 + n]);
                const float f = m[t][c] == top ? 1.f : fast_ex2(m[t][c] - top);
#pragma unroll
                for (int j = 0; j < DP / 16; ++j) {
                    ob[(warp * 8 + n) * L::OPAD + j * 16 + (lane >> 2)] = o[t][j][c] * f;
                    ob[(warp * 8 + n) * L::OPAD + j * 16 + 8 + (lane >> 2)] = o[t][j][2 + c] * f;
                }
            }
            consumer_sync();
            for (int i = threadIdx.x; ok && i < min(8, R - 8 * t) * (DP / 4); i += 32 * kConsumers) {
                const int r = i / (DP / 4), n = t * 8 + r, d = 4 * (i % (DP / 4));
                if (d >= a.dim) continue;
                float top = wm[n], sum = 0.f;
#pragma unroll
                for (int w = 1; w < kConsumers; ++w) top = fmaxf(top, wm[w * L::ROWS + n]);
                float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < kConsumers && tiles > 0; ++w) {
                    const float mw = wm[w * L::ROWS + n];
                    sum += wl[w * L::ROWS + n] * (mw == top ? 1.f : fast_ex2(mw - top));
                    const float4 y = *reinterpret_cast<const float4 *>(&ob[(w * 8 + r) * L::OPAD + d]);
                    x.x += y.x;
                    x.y += y.y;
                    x.z += y.z;
                    x.w += y.w;
                }
                if (sp.n > 1 && ctl->poisoned) {
                    x.x += poison[n * DP + d];
                    x.y += poison[n * DP + d + 1];
                    x.z += poison[n * DP + d + 2];
                    x.w += poison[n * DP + d + 3];
                }
                if (whole) {
                    const float inv = sum == 0.f ? 0.f : 1.f / sum;  // no key: zeros
                    TO *out = static_cast<TO *>(a.out) + (int64_t(sp.q0) + n / G) * a.out_token + int64_t(g * G + n % G) * a.out_head + d;
                    store4(out, x.x * inv, x.y * inv, x.z * inv, x.w * inv);
                } else {
                    const int64_t at = int64_t(walk.slot()) * plan.rows + n;
                    *reinterpret_cast<float4 *>(part_o + at * a.dim + d) = x;
                    if (d == 0) part_ml[at] = make_float2(top, sum);
                }
            }
        }
        if (tiles > 0 && ok) {
            fence_proxy_async_smem();  // the exchange lay where the next copy lands
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl->empty[kept]);
        }
    }
}

// Joins the pieces of a cut pair for one (new token, head): runs c0 .. c1 hold it, c0's
// piece in its last slot, the others' in their first.
template <typename TO>
__global__ void __launch_bounds__(32 * kJoinWarps)
rows_join_kernel(const PagedArgs a, const RowPlan plan, const float *__restrict__ part_o, const float2 *__restrict__ part_ml,
                 const int *__restrict__ starts) {
    // Before the wait: the tables.  (This block runs only once every block of the launch before has passed its own wait,
    // so whatever wrote the tables has ended.)
    const int64_t t = blockIdx.x;
    const int h = blockIdx.y, G = a.heads / a.kv_heads;
    const int b = seq_of(a.batch, t);
    bool ignore = false;
    const SeqSpan sp = b < 0 ? SeqSpan{0, 0, 0} : seq_span(a.batch, b, ignore);  // (reported by the launch before)
    const int units = tiles_of(sp, a.window, a.causal, kKeys, true).units;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (t < sp.q0 || t >= int64_t(sp.q0) + sp.n) return;
    const int share = starts[a.batch.seqs];
    const int from = starts[b] + (h / G) * units, c0 = from / share, c1 = (from + units - 1) / share;
    if (c0 == c1) return;
    const int row = int(t - sp.q0) * G + h % G;
    join_partials(a, t, h, c1 - c0 + 1, part_o, part_ml,
                  [&](int i) { return int64_t(i == 0 ? 2 * c0 + 1 : 2 * (c0 + i)) * plan.rows + row; }, static_cast<TO *>(a.out));
}

struct RowLaunch {
    RowPlan plan;
    int ctas;
};

RowLaunch row_launch(int64_t kv_heads, int64_t seqs, int64_t rows, int64_t span, int page_size) {
    RowLaunch r = {};
    r.plan.rows = int(rows);
    r.plan.box_rows = std::min(page_size & -page_size, kKeys);
    r.plan.split = span > kWholeKeys;
    const int64_t tiles = r.plan.split ? (span + kKeys - 1) / kKeys + 1 : 1;  // (a window may begin inside a tile)
    const int64_t units = seqs * kv_heads * tiles, least = r.plan.split ? kMinTiles : 1;
    r.ctas = int(std::min<int64_t>(kCtas, (units + least - 1) / least));
    return r;
}

size_t row_ws_bytes(int64_t seqs, int64_t rows, int64_t dim, int64_t ctas) {
    return size_t(2 * ctas * rows) * size_t(dim * 4 + 8) + size_t(seqs + 1) * 4;
}

template <typename T, typename TO, int DP, int NT>
cudaError_t launch_rows(const PagedArgs &a, const RowLaunch &r, const CUtensorMap &km, const CUtensorMap &vm, void *ws,
                        const LaunchCtx &ctx) {
    using L = RowLayout<DP, NT>;
    auto kernel = paged_rows_kernel<T, TO, DP, NT>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::BYTES);
    if (e != cudaSuccess) return e;
    const int64_t slots = 2 * int64_t(r.ctas) * r.plan.rows;
    float *po = r.plan.split ? static_cast<float *>(ws) : nullptr;
    float2 *pml = r.plan.split ? reinterpret_cast<float2 *>(po + slots * a.dim) : nullptr;
    int *starts = r.plan.split ? reinterpret_cast<int *>(pml + slots) : nullptr;
    e = launch_dependent(kernel, dim3(unsigned(r.ctas)), kThreads, L::BYTES, ctx.stream, km, vm, a, r.plan, po, pml, starts,
                         ctx.status, ctx.wait_ns);
    if (e != cudaSuccess || !r.plan.split) return e;
    return launch_dependent(rows_join_kernel<TO>, dim3(unsigned(a.batch.tokens), unsigned(a.heads)), 32 * kJoinWarps, 0,
                            ctx.stream, a, r.plan, po, pml, starts);
}

template <typename T, typename TO>
cudaError_t launch_rows_io(const PagedArgs &a, void *ws, const LaunchCtx &ctx) {
    const int64_t rows = int64_t(a.batch.max_q) * (a.heads / a.kv_heads);
    const int64_t span = key_span(a.batch.max_q, a.batch.max_kv, a.window);
    if (int64_t(a.batch.seqs) * a.kv_heads * (span / kKeys + 2) > INT32_MAX) return cudaErrorInvalidValue;
    const RowLaunch r = row_launch(a.kv_heads, a.batch.seqs, rows, span, a.batch.page_size);
    CUtensorMap km, vm;
    cudaError_t e = cache_maps<T>(a, r.plan.box_rows, &km, &vm);
    if (e != cudaSuccess) return e;
    if (a.dim <= 64) {
        if (rows <= 8) return launch_rows<T, TO, 64, 1>(a, r, km, vm, ws, ctx);
        if (rows <= 16) return launch_rows<T, TO, 64, 2>(a, r, km, vm, ws, ctx);
        if (rows <= 24) return launch_rows<T, TO, 64, 3>(a, r, km, vm, ws, ctx);
        return launch_rows<T, TO, 64, 4>(a, r, km, vm, ws, ctx);
    }
    if (rows <= 8) return launch_rows<T, TO, 128, 1>(a, r, km, vm, ws, ctx);
    return launch_rows<T, TO, 128, 2>(a, r, km, vm, ws, ctx);
}

}  // namespace

size_t attention_paged_ws_bytes(int64_t heads, int64_t kv_heads, int64_t dim, int64_t seqs, int64_t tokens, int64_t max_q,
                                int64_t max_kv) {
    const int64_t rows = std::min(max_q, tokens) * (heads / kv_heads);
    if (rows > rows_max(dim)) return attention_paged_chunk_ws_bytes(heads, kv_heads, dim, seqs, tokens, std::min(max_q, tokens), max_kv);
    const RowLaunch r = row_launch(kv_heads, seqs, rows, max_kv, 1);  // (a window only shortens the span)
    return r.plan.split ? row_ws_bytes(seqs, rows, dim, r.ctas) : 0;
}

cudaError_t launch_attention_paged(const PagedArgs &a, int dtype, bool out_f32, void *ws, const LaunchCtx &ctx) {
    if (int64_t(a.batch.max_q) * (a.heads / a.kv_heads) > rows_max(a.dim)) return launch_attention_paged_chunk(a, dtype, out_f32, ws, ctx);
    if (dtype == TQ2_F16) {
        if (out_f32) return launch_rows_io<__half, float>(a, ws, ctx);
        return launch_rows_io<__half, __half>(a, ws, ctx);
    }
    if (out_f32) return launch_rows_io<__nv_bfloat16, float>(a, ws, ctx);
    return launch_rows_io<__nv_bfloat16, __nv_bfloat16>(a, ws, ctx);
}

}  // namespace tq2
