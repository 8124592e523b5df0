// Grouped ternary product of a mixture of experts on the tcgen05 tensor cores:
//     out[row, f] = sum_k x[row, k] W_e[f, k]   for the rows of each expert e, or silu(gate) * up of two such.
//
// Computed transposed, W x^T: an item is 128 weight rows of one expert (the MMA's M) times a tile of up to 32, 48, 64 or 96
// staged rows of its tokens (N, any multiple of 16), so that the codes of an expert are read once for a tile of tokens
// however few they are.
//
//  * The weights never touch shared memory decoded.  A thread takes one weight row and stores its decoded weights to tensor
//    memory, which the MMA reads as its A operand.  For binary16: pairs of codes c are masked out of a word into numbers
//    2^n + c (one AND-OR a pair), less 2^n + 1 (one packed subtraction, exact).  For e4m3: four codes are looked up at a time
//    by a byte permutation.  (Left as they are masked out, as subnormal binary16 numbers, codes would cost one instruction
//    less a pair, but the tensor core aligns products by the operands' exponents: f32 sums were off by 1e-5.)
//  * The block scale d stays out of the operands: each 128-weight block is a product of its own into an accumulator of its
//    own, and d times it is added to the running sums in registers (f32).  e4m3 operands could not hold it; binary16 ones
//    could ((c - 1) d is exact for any finite d, and for code 3 below 32768, as in the dense product, which sums all of K in tensor
//    memory with 256 columns and reaches 1.2 PFLOP/s): one design serves both here, at the price of the summing groups, whose
//    registers keep a tile to 96 columns.
//  * Copies: codes by TMA, 512 weights of 128 rows a stage (96 KB in flight an SM); activations by TMA, a unit's features of a
//    tile's rows in one copy (several, of 16 rows each, took their issuing lane longer than the block's MMAs).
//  * Roles: warp 0 codes, warp 1 MMAs (owns tensor memory), warp 2 activations; two or three groups of four warps decode a
//    unit each in turn; two groups scale and sum every other item, so that one item's end (activation, staging, stores)
//    runs under the next one's blocks.  A unit is one block, or two where tiles have few columns: there the latency of
//    handing a block on is more than its work.
//    One persistent CTA an SM.  Every wait is bounded; a timeout sets the status word and the CTA drains its copies and
//    MMAs before it leaves.
//
// Bound by the roles' turns: with every copy, decoding, MMA and sum taken out, what waits and hands on still takes 175 of a
// prompt's 410 us (4096 tokens, 8 of 64 experts of 2048 x 1024, both products), and warps that poll for their turn take the
// others' issue slots (half of which are used: decoding is five instructions for eight weights of a thread's row and block
// sums are one for two).  Measured, both products: 64 tokens, 8 of 128 experts of 2048 x 768 (160 MB): 35 + 23 us, 2.7 TB/s;
// 7 tokens, 2 of 8 experts of 4096 x 6144 (160 MB): 30 + 24 us, 2.9 TB/s; the prompt 263 + 140 us, 1.02 PFLOP/s.
#include <cstdint>

#include "moe.cuh"
#include "paged_attention.cuh"

namespace tq2 {
namespace {

constexpr int W_CODES = 0, W_MMA = 1, W_ACT = 2, W_DECODE = 4;
constexpr int kCodeK = 512, kCodeBytes = 128 * kCodeK / 4;  // 16 KB
constexpr int kCodes = 6;   // stages of codes
constexpr uint32_t kTmemCols = 512;
constexpr int kMostActs = 8, kMostUnits = 4;

// COLS: 32, 64 or 96 with one or two binary16 terms, 48 with three e4m3 terms.
template <int COLS>
struct Shape {
    static constexpr bool F8 = COLS == 48, FEW = COLS <= 48;
    static constexpr int UNIT = FEW ? 2 : 1;                 // blocks that the roles hand to each other at a time
    static constexpr int RING = COLS == 64 ? 4 : 3;          // units decoded, or being multiplied
    static constexpr int DRING = COLS == 32 ? 2 : RING;      // units of accumulators: with two a unit took 400 cycles of waits
    static constexpr int ACTS = COLS == 96 ? 5 : 8;          // units of activations
    static constexpr int ACT_BYTES = COLS * kBlockW * (F8 ? 1 : 2) * UNIT;
    static constexpr int DECODERS = FEW ? 3 : 2;             // groups of four warps
    static constexpr int W_SUM = W_DECODE + 4 * DECODERS, THREADS = 32 * (W_SUM + 8);
    // registers a thread at launch, and of the roles' warpgroups after it
    static constexpr int REGS = FEW ? 80 : 96;
    static constexpr int REGS_CONTROL = FEW ? 40 : 48, REGS_DECODE = F8 ? 72 : FEW ? 80 : COLS == 64 ? 88 : 56;
    static constexpr int REGS_SUM = F8 ? 112 : FEW ? 96 : COLS == 64 ? 128 : 160;
    static constexpr int OFF_ACT = kCodes * kCodeBytes, OFF_CTL = OFF_ACT + ACTS * ACT_BYTES;
    static constexpr int A_COLS = F8 ? kBlockW / 4 : kBlockW / 2;  // of a block's decoded weights
    static constexpr uint32_t A_COL = DRING * UNIT * COLS;
    static_assert(A_COL + RING * UNIT * A_COLS <= kTmemCols, "TMEM budget");
    // (a unit's accumulators are read before its place among the units decoded is used again: no phase of `done` is missed)
    static_assert(DRING <= RING && RING <= kMostUnits && ACTS <= kMostActs);
    static_assert(REGS_CONTROL + DECODERS * REGS_DECODE + 2 * REGS_SUM <= (3 + DECODERS) * REGS, "registers");
};

struct Ctl {
    uint64_t c_full[kCodes], c_empty[kCodes];
    // by unit
    uint64_t x_full[kMostActs], x_empty[kMostActs];
    uint64_t a_full[kMostUnits];
    uint64_t done[kMostUnits];  // its MMAs have ended: its decoded weights' slot is free and its accumulators are full
    uint64_t d_empty[kMostUnits];
    uint64_t turn[2];  // a summing group may begin its next item: the other has seen all blocks of the one before
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
};
template <int COLS>
constexpr int kSmem = Shape<COLS>::OFF_CTL + int(sizeof(Ctl)) + 1024;
static_assert(kSmem<32> <= 232448 && kSmem<48> <= 232448 && kSmem<64> <= 232448 && kSmem<96> <= 232448, "shared memory budget");

__device__ __forceinline__ uint64_t desc_k(uint32_t saddr) {  // K-major, 128-byte swizzle: rows 128 B, 8-row groups 1024 B
    return uint64_t((saddr & 0x3FFFFu) >> 4) | (uint64_t(1) << 16) | (uint64_t(1024 >> 4) << 32) | (uint64_t(1) << 46) |
           (uint64_t(2) << 61);
}

__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
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

// Accumulators to registers; they are there after tm_wait_ld, and tm_tie keeps their use behind it.
__device__ __forceinline__ void tm_ld(uint32_t taddr, uint32_t (&r)[32]) {
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
__device__ __forceinline__ void tm_ld(uint32_t taddr, uint32_t (&r)[16]) { tmem_ld16(taddr, r); }
__device__ __forceinline__ void tm_wait_ld() { tc_wait_ld(); }
template <int N>
__device__ __forceinline__ void tm_tie(uint32_t (&r)[N]) {
#pragma unroll
    for (int i = 0; i < N; i += 8)
        asm volatile("" : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]), "+r"(r[i + 6]), "+r"(r[i + 7])::"memory");
}
// The same for e4m3 numbers: column c = elements 4c .. 4c + 3.
__device__ __forceinline__ void mma_ts_f8(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void tm_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
template <int N>
__device__ __forceinline__ void regs_up() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
// Two f32 at once.
__device__ __forceinline__ uint64_t pair(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ float first(uint64_t p) { return __uint_as_float(uint32_t(p)); }
__device__ __forceinline__ float second(uint64_t p) { return __uint_as_float(uint32_t(p >> 32)); }
__device__ __forceinline__ void tm_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Two words of 16 codes as 16 pairs of binary16 numbers code - 1: pair i of a word is its codes i and i + 8.  They stand at
// bits 2 i of each half; i < 5 within a binary16's mantissa, the others after a shift by 10.  The exponents are kept in
// registers: as constants beside the masks they cost an instruction more for each pair.
struct Exponents {
    uint32_t e[5];  // of 2^(10 - 2 i), in both halves: a code at bit 2 i counts ones
    __device__ __forceinline__ Exponents() {
#pragma unroll
        for (int i = 0; i < 5; ++i) asm volatile("mov.b32 %0, %1;" : "=r"(e[i]) : "r"((uint32_t(25 - 2 * i) << 10) * 0x10001u));
    }
};
__device__ __forceinline__ void decode(uint32_t w0, uint32_t w1, const Exponents &x, uint32_t (&r)[16]) {
    const uint32_t word[2] = {w0, w1};
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const uint32_t high = word[j] >> 10;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int e = i < 5 ? i : i - 5;
            uint32_t v;  // codes & mask | exponent
            asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(v) : "r"(i < 5 ? word[j] : high), "r"(0x00030003u << (2 * e)), "r"(x.e[e]));
            const __half2 s = __hsub2(*reinterpret_cast<const __half2 *>(&v), __float2half2_rn(float((1 << (10 - 2 * e)) + 1)));
            r[8 * j + i] = *reinterpret_cast<const uint32_t *>(&s);
        }
    }
}

// Four words of 16 codes as e4m3 numbers code - 1, four in a register: of each word the codes 0, 2, 4, 6, then 1, 3, 5, 7, then
// the same of its upper half, each looked up from -1, 0, 1, 2.
__device__ __forceinline__ void decode_f8(const uint4 &w, uint32_t (&r)[16]) {
    constexpr uint32_t values = 0x403800b8u;
    const uint32_t word[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t even = word[j] & 0x33333333u, odd = (word[j] >> 2) & 0x33333333u;
        r[4 * j] = __byte_perm(values, 0, even);
        r[4 * j + 1] = __byte_perm(values, 0, odd);
        r[4 * j + 2] = __byte_perm(values, 0, even >> 16);
        r[4 * j + 3] = __byte_perm(values, 0, odd >> 16);
    }
}

// Whether a phase is over, without waiting.
__device__ __forceinline__ bool phase_over(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok;
}

// Staged rows are copied by boxes of 16, 32, 64 or 96 (e4m3: 16, 32 or 48): index, and rows, of the one that holds `cols`.
template <bool F8>
__device__ __forceinline__ int box_of(int cols) { return cols <= 16 ? 0 : cols <= 32 ? 1 : F8 || cols <= 64 ? 2 : 3; }
template <bool F8>
__host__ __device__ constexpr int box_rows(int box) { return F8 ? 16 * (box + 1) : box < 3 ? 16 << box : 96; }
struct BoxMaps {
    CUtensorMap map[4];
};

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

// MMA columns of this CTA's items, one read ahead.
struct Columns {
    const MoeGemm &g;
    int parts, items, i, n;
    __device__ __forceinline__ Columns(const MoeGemm &gemm, int p, int count) : g(gemm), parts(p), items(count), i(blockIdx.x) { read(); }
    __device__ __forceinline__ void read() { n = i < items ? g.plan.tiles[i / parts].n : 0; }
    __device__ __forceinline__ int take() {
        const int cols = (n * g.terms + 15) & ~15;
        i += gridDim.x;
        read();
        return cols;
    }
};

// x / (1 + exp(-x)).  EXACT (f32 layers; gates are cut off at 87 on either side): exp by the hardware's 2^t of the rounded exponent,
// times 1 + what the rounding left of it, the reciprocal with one Newton step: 2 units in the last place and 1.  (expf and a
// division took a chunk of 513 tokens from 76 to 83 us: an item's end is straight code that is fetched each time.)
// Else by the fast exponential, within 2 + 1.173 |x| units in the last place, and the fast quotient, within 2 (and 0 below
// -87.3): 2^-18 at -24, of values that go on in 11 or 12 bits (EXACT there: a prompt of 4096 tokens 531 -> 550 us).
template <bool EXACT>
__device__ __forceinline__ float silu(float x) {
    if (!EXACT) return __fdividef(x, 1.f + __expf(-x));
    constexpr float l_hi = 1.44269502f, l_lo = 1.92596303e-8f, ln2 = 0.69314718f;  // log2(e) in two parts
    const float z = fminf(fmaxf(x, -87.f), 87.f), t = z * -l_hi;
    const float rest = fmaf(z, -l_lo, fmaf(z, -l_hi, -t)), p = fast_ex2(t);
    const float y = 1.f + fmaf(p, rest * ln2, p);
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(y));
    return x * fmaf(r, fmaf(-y, r, 1.f), r);
}

template <bool GATE_UP, int COLS>
__global__ void __launch_bounds__(Shape<COLS>::THREADS, 1)
moe_gemm_kernel(const __grid_constant__ CUtensorMap cmap, const __grid_constant__ BoxMaps xmaps, const MoeGemm g,
                unsigned int *status, uint64_t wait_ns) {
    using L = Shape<COLS>;
    extern __shared__ __align__(1024) uint8_t raw[];
    uint8_t *smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    Ctl *ctl = reinterpret_cast<Ctl *>(smem + L::OFF_CTL);
    const int warp = uniform(int(threadIdx.x >> 5)), lane = threadIdx.x & 31;
    volatile int *abort_flag = &ctl->abort;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kCodes; ++s) {
            mbar_init(&ctl->c_full[s], 1);
            mbar_init(&ctl->c_empty[s], 4 * L::DECODERS);
        }
        for (int s = 0; s < L::ACTS; ++s) {
            mbar_init(&ctl->x_full[s], 1);
            mbar_init(&ctl->x_empty[s], 1);
        }
        for (int s = 0; s < L::RING; ++s) {
            mbar_init(&ctl->a_full[s], 4);
            mbar_init(&ctl->done[s], 1);
        }
        for (int s = 0; s < L::DRING; ++s) mbar_init(&ctl->d_empty[s], 4);
        for (int s = 0; s < 2; ++s) mbar_init(&ctl->turn[s], 4);
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
    const int parts = g.rows / 128, nb = uniform(g.k / kBlockW), units = (nb + L::UNIT - 1) / L::UNIT;
    const int items = uniform(*g.plan.tile_count * parts);
    auto wait_on = [&](uint64_t *bar, uint32_t parity, uint32_t first_poll = 0) {
        return bool(__all_sync(0xffffffffu, wait_phase(bar, parity, abort_flag, wait_ns, status, first_poll)));
    };

    if (warp < W_DECODE) {
        regs_down<L::REGS_CONTROL>();
        if (warp == W_CODES) {
            int n = 0;  // stages filled
            bool ok = true;
            for (int i = blockIdx.x; ok && i < items; i += gridDim.x) {
                const Item it = item_of(g, i, parts);
                const int row = it.tile.expert * g.rows;
                const int y0 = row + (GATE_UP ? 64 : 128) * it.part, y1 = GATE_UP ? y0 + g.rows / 2 : y0 + 64;
                for (int k = 0; k < g.k; k += kCodeK, ++n) {
                    const int s = n % kCodes;
                    if (n >= kCodes && !(ok = wait_on(&ctl->c_empty[s], (n / kCodes - 1) & 1))) break;
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
                for (int j = max(0, n - kCodes); j < n; ++j)
                    mbar_wait_bounded(&ctl->c_full[j % kCodes], (j / kCodes) & 1, drain_ns(wait_ns), status);
            __syncwarp();
        } else if (warp == W_ACT) {
            int n = 0;
            bool ok = true;
            for (int i = blockIdx.x; ok && i < items; i += gridDim.x) {
                const Item it = item_of(g, i, parts);
                // (one copy a unit, issued by one lane: its issue takes longer than the block's MMAs; the box's rows after the
                // tile's are other experts', whose columns nothing reads)
                const int box = uniform(box_of<L::F8>(it.cols)), bytes = box_rows<L::F8>(box) * (L::F8 ? 128 : 256) * L::UNIT, row = it.tile.row0 * g.terms;
                for (int u = 0; u < units; ++u, ++n) {
                    const int s = n % L::ACTS;
                    if (!(ok = wait_on(&ctl->x_empty[s], ((n / L::ACTS) & 1) ^ 1))) break;
                    if (elect_one()) {
                        mbar_expect_tx(&ctl->x_full[s], uint32_t(bytes));
                        tma_3d(smem_u32(smem) + uint32_t(L::OFF_ACT + s * L::ACT_BYTES), &xmaps.map[box], 0, row,
                               u * L::UNIT * (L::F8 ? 1 : 2), &ctl->x_full[s]);
                    }
                    __syncwarp();
                }
            }
            if (lane == 0)
                for (int j = max(0, n - L::ACTS); j < n; ++j)
                    mbar_wait_bounded(&ctl->x_full[j % L::ACTS], (j / L::ACTS) & 1, drain_ns(wait_ns), status);
            __syncwarp();
        } else if (warp == W_MMA) {
            // (the whole warp takes the loop, from values that the compiler knows to be uniform, and one lane issues)
            const uint64_t x0 = desc_k(smem_u32(smem) + uint32_t(L::OFF_ACT));
            int n = 0;  // units
            bool ok = true;
            Columns next(g, parts, items);
            for (int i = blockIdx.x; ok && i < items; i += gridDim.x) {
                const int cols = uniform(next.take());
                const uint32_t idesc = (1u << 4) | (uint32_t(cols >> 3) << 17) | (uint32_t(128 >> 4) << 24);
                const uint32_t piece = uint32_t(box_rows<L::F8>(box_of<L::F8>(cols))) * 8;  // (in 16 bytes) 128 bytes of each of the box's rows
                for (int u = 0; u < units; ++u, ++n) {
                    const int s = n % L::RING, sx = n % L::ACTS, sd = n % L::DRING;
                    // (asked for together: one after the other the answers took 300 cycles a block; a slot's phase before
                    // its first use counts as over)
                    const uint32_t pd = ((n / L::DRING) & 1) ^ 1, px = (n / L::ACTS) & 1, pa = (n / L::RING) & 1;
                    for (int polls = 0; ok; ++polls) {
                        const bool d_free = phase_over(&ctl->d_empty[sd], pd), x_there = phase_over(&ctl->x_full[sx], px),
                                   a_there = phase_over(&ctl->a_full[s], pa);
                        if (__all_sync(0xffffffffu, d_free && x_there && a_there)) break;
                        if (polls == 4)
                            ok = wait_on(&ctl->d_empty[sd], pd) && wait_on(&ctl->x_full[sx], px) && wait_on(&ctl->a_full[s], pa);
                        if (polls == 4) break;
                    }
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t dx = x0 + uint64_t(uint32_t(sx) * (L::ACT_BYTES >> 4));
                    const uint32_t d = tmem + uint32_t(sd * L::UNIT * COLS), at = tmem + L::A_COL + uint32_t(s * L::UNIT * L::A_COLS);
                    const bool both = u * L::UNIT + L::UNIT <= nb;
                    if (elect_one()) {
#pragma unroll
                        for (int j = 0; j < L::UNIT; ++j) {
                            if (j > 0 && !both) break;
                            const uint64_t db = dx + uint64_t((L::F8 ? 1 : 2) * j * piece);
#pragma unroll
                            for (int kk = 0; kk < (L::F8 ? 4 : 8); ++kk)
                                if (L::F8)
                                    mma_ts_f8(d + j * COLS, at + uint32_t(j * L::A_COLS + kk * 8), db + uint64_t(2 * kk), idesc, kk > 0);
                                else
                                    mma_ts(d + j * COLS, at + uint32_t(j * L::A_COLS + kk * 8),
                                           db + uint64_t((kk >> 2) * piece + 2 * (kk & 3)), idesc, kk > 0);
                        }
                        tc_commit(&ctl->done[s]);
                        tc_commit(&ctl->x_empty[sx]);
                    }
                    __syncwarp();
                }
            }
            if (elect_one()) tc_commit(&ctl->drain);
            __syncwarp();
        }
    } else if (warp < L::W_SUM) {
        regs_down<L::REGS_DECODE>();
        const int q = warp & 3, group = (warp - W_DECODE) >> 2;
        // the row of this thread's lane among the stage's 128: gate rows in lanes 0-15, the up rows of the same features above
        const int r = GATE_UP ? (lane < 16 ? 16 * q + lane : 48 + 16 * q + lane) : 32 * q + lane;
        // This group's units are every other one, or third, of all.  Each group waits for every stage of codes, so that none is
        // ever two uses of a slot ahead of another.
        const Exponents exponents;
        constexpr int DEC = L::DECODERS, PER = 4 / L::UNIT, MINE = (PER + DEC - 1) / DEC;  // units of a stage, and of them a group's
        int n0 = 0, stage0 = 0;  // units and stages before the item
        bool ok = true;
        for (int i = blockIdx.x; ok && i < items; i += gridDim.x, n0 += units, stage0 += (nb + 3) / 4) {
            for (int u0 = 0; ok && u0 < units; u0 += PER) {
                const int stage = stage0 + u0 / PER, sc = stage % kCodes;
                if (!(ok = wait_on(&ctl->c_full[sc], (stage / kCodes) & 1))) break;
                const uint8_t *row = smem + sc * kCodeBytes + r * 128;
                const int from = (group + DEC - (n0 + u0) % DEC) % DEC;  // this group's first unit of the stage (or of a later one)
                uint4 w[MINE][L::UNIT][2];
#pragma unroll
                for (int t = 0; t < MINE; ++t)
#pragma unroll
                    for (int j = 0; j < L::UNIT; ++j)
#pragma unroll
                        for (int c = 0; c < 2; ++c)
                            w[t][j][c] = *reinterpret_cast<const uint4 *>(
                                row + (((2 * (min(from + DEC * t, PER - 1) * L::UNIT + j) + c) ^ (r & 7)) << 4));
                // (read before the next copy may write there: without it loads were put off to where the codes are decoded, behind
                // the wait for a slot, and where codes came late from memory some rows had the next stage's)
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl->c_empty[sc]);
#pragma unroll
                for (int t = 0; t < MINE; ++t) {
                    const int u = u0 + from + DEC * t, n = n0 + u, s = n % L::RING;
                    if (from + DEC * t >= PER || u >= units) break;
                    if (!(ok = wait_on(&ctl->done[s], ((n / L::RING) & 1) ^ 1))) break;
                    tc_fence_after();
#pragma unroll
                    for (int j = 0; j < L::UNIT; ++j) {
                        if (u * L::UNIT + j >= nb) break;
                        const uint32_t at = tmem + L::A_COL + uint32_t((s * L::UNIT + j) * L::A_COLS) + (uint32_t(q * 32) << 16);
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            if (L::F8) {
                                uint32_t v[16];
                                decode_f8(w[t][j][c], v);
                                tm_st16(at + uint32_t(16 * c), v);
                                continue;
                            }
                            // (stores of 16 registers: of 32, the next ones waited for these to be read)
                            uint32_t v[2][16];
                            decode(w[t][j][c].x, w[t][j][c].y, exponents, v[0]);
                            tm_st16(at + uint32_t(32 * c), v[0]);
                            decode(w[t][j][c].z, w[t][j][c].w, exponents, v[1]);
                            tm_st16(at + uint32_t(32 * c + 16), v[1]);
                        }
                    }
                    tm_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ctl->a_full[s]);
                }
            }
        }
    } else {
        regs_up<L::REGS_SUM>();
        const int q = warp & 3, group = (warp - L::W_SUM) >> 2;
        const int features = GATE_UP ? g.rows / 2 : g.rows;
        int n0 = group * units, turn = group;  // units and items of this CTA before the item
        bool ok = true;
        for (int i = blockIdx.x + group * gridDim.x; ok && i < items; i += 2 * gridDim.x, n0 += 2 * units, turn += 2) {
            const Item it = item_of(g, i, parts);
            const int row = it.tile.expert * g.rows + (GATE_UP ? 64 * it.part + 16 * q + (lane & 15) + (lane < 16 ? 0 : g.rows / 2)
                                                              : 128 * it.part + 32 * q + lane);
            const __half *dp = g.d + int64_t(row) * nb;
            // the scales of the tile's rows, some in each lane
            const int left = it.tile.n;
            float scale[COLS / 32], up[COLS / 32];  // up (gate_up): the power of two that the hidden values are staged with
            float sum_x[COLS / 32], peak_x[COLS / 32];
            constexpr bool STAGES = GATE_UP && !L::F8;
#pragma unroll
            for (int j = 0; j < COLS / 32; ++j) {
                const int at = it.tile.row0 + min(32 * j + lane, left - 1);
                scale[j] = g.scale[at];
                if (STAGES) {
                    sum_x[j] = g.sum[at];
                    peak_x[j] = g.peak[at];
                }
            }
            if (STAGES) {
                uint32_t most = 0, whole = 0;
                for (int j = lane; j < g.bound_blocks; j += 32) {
                    const float2 b = g.plan.bound[it.tile.expert * g.bound_blocks + j];
                    most = max(most, __float_as_uint(b.x));
                    whole = max(whole, __float_as_uint(b.y));
                }
                most = __reduce_max_sync(0xffffffffu, most);
                whole = __reduce_max_sync(0xffffffffu, whole);
#pragma unroll
                for (int j = 0; j < COLS / 32; ++j) {
                    // |h| <= b^2 < 2^(2 e + 2) (see moe.cuh), so that times 2^(13 - 2 e) it is below 2^15
                    const float b = 2.f * fminf(__uint_as_float(most) * sum_x[j], __uint_as_float(whole) * peak_x[j]);
                    const int e = b < INFINITY ? max(min(13 - 2 * moe_log2(b), 126), -126) : 0;
                    up[j] = moe_power(e);
                    if (it.part == 0 && q == 0) g.scale_out[it.tile.row0 + min(32 * j + lane, left - 1)] = moe_power(-e);
                }
            }
            uint64_t acc[COLS / 2];  // columns 2 c, 2 c + 1
#pragma unroll
            for (int c = 0; c < COLS / 2; ++c) acc[c] = 0;
            float dn[L::UNIT];
            auto scales_of = [&](int u) {
#pragma unroll
                for (int j = 0; j < L::UNIT; ++j) dn[j] = u * L::UNIT + j < nb ? __half2float(dp[u * L::UNIT + j]) : 0.f;
            };
            scales_of(0);
            // (in turn: a group that waited for a unit two uses of its accumulator ahead would take the one before for it; the
            // longest wait of all, which a limit of 0 gives up after one poll: looked at in all of them, that took a prompt
            // from 530 to 534 us)
            if (turn > 0 && !(ok = wait_on(&ctl->turn[group], ((turn - 1) >> 1) & 1, wait_ns ? 0 : 63))) break;
            for (int u = 0; u < units; ++u) {
                const int n = n0 + u, sd = n % L::DRING;
                uint64_t d[L::UNIT];
#pragma unroll
                for (int j = 0; j < L::UNIT; ++j) d[j] = pair(dn[j], dn[j]);
                scales_of(u + 1);
                if (!(ok = wait_on(&ctl->done[n % L::RING], (n / L::RING) & 1))) break;
                tc_fence_after();
                const uint32_t at = tmem + uint32_t(sd * L::UNIT * COLS) + (uint32_t(q * 32) << 16);
                const bool both = u * L::UNIT + L::UNIT <= nb;
                // 32 values in flight: 32 columns of a block, or 16 of each of two
                constexpr int W = 32 / L::UNIT;
#pragma unroll
                for (int h = 0; h < COLS / W; ++h)
                    if (W * h < it.cols) {
                        uint32_t v[L::UNIT][W];
#pragma unroll
                        for (int j = 0; j < L::UNIT; ++j) {
                            if (j > 0 && !both) {
#pragma unroll
                                for (int c = 0; c < W; ++c) v[j][c] = 0;
                            } else {
                                tm_ld(at + uint32_t(j * COLS + W * h), v[j]);
                            }
                        }
                        tm_wait_ld();
#pragma unroll
                        for (int j = 0; j < L::UNIT; ++j) {
                            tm_tie(v[j]);
#pragma unroll
                            for (int c = 0; c < W / 2; ++c)
                                acc[W / 2 * h + c] =
                                    fma2(d[j], uint64_t(v[j][2 * c]) | uint64_t(v[j][2 * c + 1]) << 32, acc[W / 2 * h + c]);
                        }
                    }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl->d_empty[sd]);
            }
            if (!ok) break;
            if (lane == 0) mbar_arrive(&ctl->turn[group ^ 1]);
            auto finish = [&](auto two) {
                constexpr int S = decltype(two)::value;
                // row c of the tile: column c, or the sum of the columns of its terms
                auto column = [&](int c) { return c & 1 ? second(acc[c >> 1]) : first(acc[c >> 1]); };
                auto sum = [&](int c) {
                    if (S == 3) return fmaf(fmaf(column(3 * c + 2), 0x1p-4f, column(3 * c + 1)), 0x1p-4f, column(3 * c));
                    return S == 2 ? fmaf(column(2 * c + 1), 1.f / kLowScale, column(2 * c)) : column(c);
                };
                if (GATE_UP) {
                    // this lane's place in a staged row
                    __half *out = g.staged_out + int64_t(it.tile.row0) * S * features + 64 * it.part + 16 * q + moe_place(lane & 15);
                    float *plain = g.out + int64_t(it.tile.row0) * features + 64 * it.part + 16 * q + (lane & 15);
                    const int odd = lane >= 16;
#pragma unroll
                    for (int c0 = 0; c0 < COLS / S; c0 += 8)
                        if (c0 < left) {
                            // lanes 0-15 finish row c, lanes 16-31 row c + 1 (four of them together: one's steps wait for each other)
                            float gate[4], ups[4], by[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int c = c0 + 2 * i;
                                const float s = __shfl_sync(0xffffffffu, scale[c >> 5], (c & 31) + odd);
                                by[i] = S == 3 ? 1.f : __shfl_sync(0xffffffffu, up[c >> 5], (c & 31) + odd);
                                const float other = __shfl_xor_sync(0xffffffffu, odd ? sum(c) : sum(c + 1), 16);
                                gate[i] = (odd ? other : sum(c)) * s;
                                ups[i] = (odd ? sum(c + 1) : other) * s;
                            }
#pragma unroll
                            for (int i = 0; i < 4; ++i) gate[i] = silu<S == 2>(gate[i]) * ups[i] * by[i];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int row = c0 + 2 * i + odd;
                                if (row >= left) continue;
                                const float h = gate[i];
                                if (S == 3) {
                                    plain[int64_t(row) * features] = h;
                                } else {
                                    const __half hi = __float2half_rn(h);
                                    __half *to = out + int64_t(row) * S * features;
                                    to[0] = hi;
                                    if (S == 2) to[features] = __float2half_rn((h - __half2float(hi)) * kLowScale);
                                }
                            }
                        }
                } else {
                    float *out = g.out + int64_t(it.tile.row0) * features + 128 * it.part + 32 * q + lane;
#pragma unroll
                    for (int c0 = 0; c0 < COLS / S; c0 += 8)
                        if (c0 < left) {
#pragma unroll
                            for (int c = c0; c < c0 + 8; ++c) {
                                const float s = __shfl_sync(0xffffffffu, scale[c >> 5], c & 31);
                                if (c < left) out[int64_t(c) * features] = sum(c) * s;
                            }
                        }
                }
            };
            if (L::F8)
                finish(std::integral_constant<int, 3>{});
            else if (g.terms == 2)
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

cudaError_t make_map(CUtensorMap *map, CUtensorMapDataType type, const void *base, int rank, const cuuint64_t *dims,
                     const cuuint64_t *strides, const cuuint32_t *box, CUtensorMapL2promotion promote) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return cudaErrorNotSupported;
    const cuuint32_t step[3] = {1, 1, 1};
    if (enc(map, type, cuuint32_t(rank), const_cast<void *>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, promote, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    return cudaSuccess;
}

template <int COLS>
cudaError_t launch(const MoeGemm &g, bool gate_up, const LaunchCtx &ctx) {
    CUtensorMap cmap;
    BoxMaps xmaps = {};
    const cuuint64_t cdims[2] = {cuuint64_t(g.k / 4), cuuint64_t(g.experts) * cuuint64_t(g.rows)}, cstrides[1] = {cuuint64_t(g.k / 4)};
    const cuuint32_t cbox[2] = {128, 64};
    cudaError_t e = make_map(&cmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, g.qs, 2, cdims, cstrides, cbox, CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
    // [128-byte pieces of a row][rows][a piece]: a unit's pieces in one copy, each a swizzled operand
    constexpr bool F8 = Shape<COLS>::F8;
    constexpr int size = F8 ? 1 : 2, piece = 128 / size;
    const cuuint64_t xdims[3] = {piece, cuuint64_t(g.pairs * g.terms), cuuint64_t(g.k / piece)};
    const cuuint64_t xstrides[2] = {cuuint64_t(g.k) * size, 128};
    for (int i = 0; i < 4 && box_rows<F8>(i) <= COLS && e == cudaSuccess; ++i) {
        const cuuint32_t xbox[3] = {piece, cuuint32_t(box_rows<F8>(i)), cuuint32_t(kBlockW / piece * Shape<COLS>::UNIT)};
        e = make_map(&xmaps.map[i], F8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, g.staged, 3, xdims, xstrides,
                     xbox, CU_TENSOR_MAP_L2_PROMOTION_L2_128B);
    }
    if (e != cudaSuccess) return e;
    auto kernel = gate_up ? moe_gemm_kernel<true, COLS> : moe_gemm_kernel<false, COLS>;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem<COLS>);
    if (e != cudaSuccess) return e;
    const int64_t items = int64_t(g.max_tiles) * (g.rows / 128);
    const unsigned grid = unsigned(std::min<int64_t>(items, ctx.num_sms));
    return launch_dependent(kernel, dim3(grid), Shape<COLS>::THREADS, kSmem<COLS>, ctx.stream, cmap, xmaps, g, ctx.status, ctx.wait_ns);
}

}  // namespace

cudaError_t launch_moe_gemm(const MoeGemm &g, bool gate_up, const LaunchCtx &ctx) {
    switch (g.cols) {
        case 32: return launch<32>(g, gate_up, ctx);
        case 48: return launch<48>(g, gate_up, ctx);
        case 64: return launch<64>(g, gate_up, ctx);
        default: return launch<96>(g, gate_up, ctx);
    }
}

}  // namespace tq2
