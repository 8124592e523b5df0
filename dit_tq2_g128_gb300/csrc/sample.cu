// Sampling: one token of each row of logits, by a given random number.
//
// Tokens are ordered by their logits, descending, equal ones by index.  Weights w = exp((l - max) / temperature) are
// integers in units of 2^-45 (sample_weight.cuh), so that sums of them are exact in any order; top-k, top-p and min-p
// each keep a prefix of the order, and the token drawn is the first whose cumulative weight passes u times the kept
// weight.  Every question is then one of a count or a sum over a prefix, and no sort of a row is needed.
//
// A cluster of CTAs takes a row and keeps it in shared memory: it is read from memory once.
//  * With a top-k of up to 768 (and of rows of up to 1024 logits, or of which only the largest weigh anything), the head: a
//    bound that at least k of the maxima of groups of threads reach; the few elements above it go to the first CTA, which
//    sorts them and answers every question from their cumulative weights.
//  * Without a top-k, a guess: a histogram of counts (5888 bins of log2 of the weight, their elements taken to lie in the middle)
//    says within some elements where top_p's border and the drawn token lie.  One pass then adds up the exact weights of all
//    elements and of those above either place, and collects the few about them, which are sorted; if the exact prefixes pass
//    their targets among these, they are the answer.
//  * Else (a larger k, many equal logits, a guess that failed): a histogram of counts and exact weights finds the bin that an
//    answer lies in; its elements (at most 1024, or split further by their bits) are sorted as the head is.
//
// Bound by latency for one row (32,000 logits: 8.1 us) and by a row's chain for many: with a top-k 28,000 cycles (loading 9,
// four cluster barriers with the bound 6, collecting 5, sorting 5, the answer 3), two CTAs an SM (256 rows of 100,003
// bf16 logits: 63 us); without one 55,000, of which the exact sums are a third, some 60 instructions a weight (16 flat rows of
// 200,000: 40 us; 64 rows of 128,000 f32, a quarter without a top-k: 49 us, all: 71, of bf16 53, all with one of 2000: 92; one
// such row 22).  The exact histogram in place of the guess, with
// four shared atomics an element and two passes to collect, took 81 and 75 us.  64 registers a thread, so that two CTAs share
// an SM: 4 bytes a thread are spilled and read 32 times (bf16: 52 bytes, 42 times; by the compiler's count).
#include <algorithm>
#include <cstdint>

#include "cluster.cuh"
#include "dtype.cuh"
#include "paged_attention.cuh"
#include "sample_weight.cuh"
#include "tq2_internal.cuh"

namespace tq2 {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBins = 1472;  // of y: 32 or more in a unit (of log2 of the weight)
constexpr int kFine = 4 * kBins;  // of y in a guess, in the same memory
constexpr int kList = 1024;
constexpr int kMostHeadK = 768, kRankSort = 256;
constexpr int kEach = kList / kThreads;  // list elements of a thread
constexpr int kMaxCluster = 8;
static_assert(kBins % (4 * kMaxCluster) == 0);

enum Op { OP_DONE, OP_HISTOGRAM, OP_REFINE, OP_SPAN, OP_GATHER, OP_HEAVY, OP_TIE };
// What the first CTA has the others do.
struct Command {
    int op, bin, shift;
    uint32_t low, high;  // keys
    uint32_t rank;       // OP_TIE: which of the elements `low`, from 0
};

struct alignas(16) Shared {  // (the row follows it, in packs of 16 bytes)
    // Weights of bins.  While they are counted, in three pieces of 15 bits and more (a 64-bit atomic is a loop here, and
    // 2^15 of a piece fit 32 bits); then, in the first CTA, the low and the high word of their sum over the CTAs.
    uint32_t mass[3][kBins], count[kBins];
    unsigned long long list[kList];  // key << 32 | ~index
    unsigned long long cum[kList];
    uint64_t table[64];
    unsigned long long part[kWarps];
    unsigned long long total, found_mass, found_before, kept;
    unsigned long long sums[4], my_sums[4];  // of a guess: all weights, those min_p keeps, those above each range; this CTA's
    float range[2][2];  // logits from and to which answers are looked for
    float heavy[2];  // what min_p keeps, without and with the bin it ends in
    int edge[4];
    uint32_t until[4];
    uint32_t top[kMaxCluster], ties[kMaxCluster];
    float bottom[kMaxCluster];
    uint32_t n_list, n_mine, base, low, high;
    int found;
    float floor;  // the head: logits from here on
    Command cmd;
};

__device__ __forceinline__ unsigned long long warp_scan(unsigned long long v) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long x = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += x;
    }
    return v;
}
// Inclusive sums over the block's threads.
__device__ __forceinline__ unsigned long long block_scan(unsigned long long v, Shared *sh) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    v = warp_scan(v);
    __syncthreads();
    if (lane == 31) sh->part[warp] = v;
    __syncthreads();
    if (warp == 0) {
        const unsigned long long s = warp_scan(lane < kWarps ? sh->part[lane] : 0);
        if (lane < kWarps) sh->part[lane] = s;
    }
    __syncthreads();
    return v + (warp ? sh->part[warp - 1] : 0);
}

// A bitonic network of E elements a thread in registers (i, and i + kThreads), whose steps within a warp are shuffles.
template <int E>
__device__ __forceinline__ void sort_network(unsigned long long *list, unsigned long long *spare, int count) {
    const int i = threadIdx.x;
    unsigned long long v[E];
#pragma unroll
    for (int j = 0; j < E; ++j) v[j] = i + j * kThreads < count ? list[i + j * kThreads] : 0;
    auto keep = [&](int j, unsigned long long other, int step, bool falling) {
        v[j] = ((i & step) == 0) == falling ? max(v[j], other) : min(v[j], other);
    };
    auto within = [&](int step, int size) {
#pragma unroll
        for (int j = 0; j < E; ++j) keep(j, __shfl_xor_sync(0xffffffffu, v[j], step), step, ((i + j * kThreads) & size) == 0);
    };
#pragma unroll
    for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
        for (int step = size >> 1; step; step >>= 1) within(step, size);
    bool odd = false;
#pragma unroll 1
    for (int size = 64; size <= E * kThreads; size <<= 1) {
        int step = size >> 1;
        if (E == 2 && step == kThreads) {
            const unsigned long long top = max(v[0], v[E - 1]), low = min(v[0], v[E - 1]);
            v[0] = top;
            v[E - 1] = low;
            step >>= 1;
        }
#pragma unroll 1
        for (; step >= 32; step >>= 1) {
            unsigned long long *to = odd ? spare : list;  // (in turn, so that one barrier a step is enough)
            odd = !odd;
#pragma unroll
            for (int j = 0; j < E; ++j) to[i + j * kThreads] = v[j];
            __syncthreads();
#pragma unroll
            for (int j = 0; j < E; ++j) keep(j, to[(i ^ step) + j * kThreads], step, ((i + j * kThreads) & size) == 0);
        }
#pragma unroll
        for (step = 16; step; step >>= 1) within(step, size);
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < E; ++j) list[i + j * kThreads] = v[j];
    __syncthreads();
}
// Sorts list[0, count) descending (all different).  Short ones by counting who is larger (a list of 100: 700 cycles, not
// the 5000 of a network's 28 steps through shared memory); others by a bitonic network of one or two elements a thread, in
// registers, whose steps within a warp are shuffles (of 400: 7,000 cycles, not 11,000 through shared memory).
__device__ __forceinline__ void sort_list(unsigned long long *list, unsigned long long *spare, int count) {
    const int i = threadIdx.x;
    if (count <= kRankSort) {
        __syncthreads();
        if (i < count) {
            const unsigned long long mine = list[i];
            int larger = 0;
#pragma unroll 4
            for (int j = 0; j < count; ++j) larger += list[j] > mine;
            spare[larger] = mine;
        }
        __syncthreads();
        if (i < count) list[i] = spare[i];
        __syncthreads();
        return;
    }
    if (count <= kThreads)
        sort_network<1>(list, spare, count);
    else
        sort_network<2>(list, spare, count);
}

// A pack of 16 bytes.
template <typename T>
struct alignas(16) Pack {
    static constexpr int N = 16 / sizeof(T);
    T e[N];
};
// Elements src[0, n) to x[0, n), both at the same place in a pack.  Returns the thread's largest (-inf where it has none);
// lowest: its smallest above -inf (inf).
template <typename T>
__device__ __forceinline__ float load_slice(const T *src, int n, T *x, float *lowest) {
    constexpr int V = Pack<T>::N, U = 4;
    const int shift = int(reinterpret_cast<uintptr_t>(src) & 15) / int(sizeof(T));
    const Pack<T> *from = reinterpret_cast<const Pack<T> *>(src - shift);
    Pack<T> *to = reinterpret_cast<Pack<T> *>(x - shift);
    const int packs = n > 0 ? (n + shift + V - 1) / V : 0;
    const T nan = from_f32<T>(__uint_as_float(0x7fc00000u));
    float best = -INFINITY, least = INFINITY;
    for (int p0 = threadIdx.x; p0 < packs; p0 += U * kThreads) {
        Pack<T> v[U];
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int p = p0 + j * kThreads;
            if (p > 0 && p < packs - 1)
                v[j] = from[p];
            else if (p < packs)  // (nothing outside the row is read)
                for (int i = 0; i < V; ++i) {
                    const int at = p * V + i - shift;
                    v[j].e[i] = at >= 0 && at < n ? src[at] : nan;
                }
        }
#pragma unroll
        for (int j = 0; j < U; ++j)
            if (p0 + j * kThreads < packs) {
                to[p0 + j * kThreads] = v[j];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float f = to_f32(v[j].e[i]);
                    best = fmaxf(best, f);
                    least = f > -INFINITY ? fminf(least, f) : least;
                }
            }
    }
    *lowest = least;
    return best;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(SampleArgs a, int slice, int cluster) {
    extern __shared__ __align__(16) uint8_t raw[];
    Shared *sh = reinterpret_cast<Shared *>(raw);
    const int tid = threadIdx.x, lane = tid & 31;
    const uint32_t rank = cluster_rank();
    const int64_t r = blockIdx.x / cluster;
    Shared *lead = at_cta(sh, 0);
    cluster_arrive();  // (begun; waited for before another CTA's memory is written, behind the row's load)
    uint32_t *fine = sh->mass[0];
    for (int i = tid; i < kFine; i += kThreads) fine[i] = 0;
    if (tid < 4) sh->sums[tid] = sh->my_sums[tid] = 0;
    if (tid < 64) sh->table[tid] = weight_table.e[tid];
    if (tid == 0) {
        sh->n_list = 0;
        sh->n_mine = 0;
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // ---- the row, and its largest logit
    const int first = int(rank) * slice, n = max(0, min(slice, a.vocab - first));
    const float temperature = a.temperature ? a.temperature[r] : 1.f, p = a.top_p ? a.top_p[r] : 1.f, u = a.u[r];
    const int k = a.top_k ? a.top_k[r] : 0;
    const uint64_t least = a.min_p ? least_weight(a.min_p[r]) : 0;
    const T *src = static_cast<const T *>(a.logits) + r * a.row_stride + first;
    constexpr int V = Pack<T>::N;
    const int shift = int(reinterpret_cast<uintptr_t>(src) & 15) / int(sizeof(T));
    T *x = reinterpret_cast<T *>(raw + sizeof(Shared)) + shift;
    float lowest;
    const float mine = load_slice(src, n, x, &lowest);
    {
        const uint32_t m = __reduce_max_sync(0xffffffffu, order_key(mine));
        const uint32_t l = __reduce_min_sync(0xffffffffu, order_key(lowest));
        if (lane == 0) sh->part[tid >> 5] = static_cast<unsigned long long>(l) << 32 | m;
        __syncthreads();
        cluster_wait();  // every CTA has begun
        if (tid < cluster) {
            uint32_t best = 0, least = 0xffffffffu;
            for (int w = 0; w < kWarps; ++w) {
                best = max(best, uint32_t(sh->part[w]));
                least = min(least, uint32_t(sh->part[w] >> 32));
            }
            at_cta(sh, uint32_t(tid))->top[rank] = best;
            at_cta(sh, uint32_t(tid))->bottom[rank] = key_value(least);
        }
    }
    cluster_sync();
    uint32_t top = 0;
    float bottom = INFINITY;
    for (int c = 0; c < cluster; ++c) {
        top = max(top, sh->top[c]);
        bottom = fminf(bottom, sh->bottom[c]);
    }
    if (top <= order_key(-INFINITY)) {  // nothing left
        if (rank == 0 && tid == 0) {
            a.tokens[r] = -1;
            if (a.prob) a.prob[r] = 0.f;
        }
        return;
    }
    const RowWeights rw(key_value(top), temperature);
    // The bin of a logit; -1: no weight.  The bins share out what y the row has.
    const float most = fminf(rw.coarse(bottom), float(kWeightBits + 1));
    const float per_unit = most > 0.f ? fminf(float(kBins - 1) / most, 1e6f) : 1.f;
    auto bin_of_logit = [&](float l) {
        const float y = rw.coarse(l);
        return y < float(kWeightBits + 1) ? min(int(y * per_unit), kBins - 1) : -1;
    };
    const bool cut_k = k > 0 && k < a.vocab, cut_p = p < 1.f;

    // f(value) for all elements, a pack at a time (and for the NaNs that fill the first and last packs)
    const Pack<T> *packed = reinterpret_cast<const Pack<T> *>(x - shift);
    const int packs = n > 0 ? (n + shift + V - 1) / V : 0;
    auto each = [&](auto f) {
        for (int q = tid; q < packs; q += kThreads) {
            const Pack<T> v = packed[q];
#pragma unroll
            for (int i = 0; i < V; ++i) f(to_f32(v.e[i]));
        }
    };
    // The elements that are `wanted` to the first CTA's list: marked, placed in this CTA's own by one count a warp, and handed
    // over all at once.  (Taken one by one, with a count each, they were a third of a row's time.)
    auto collect = [&](bool look, auto wanted) {
        for (int q0 = 0; q0 < packs; q0 += 64 / V * kThreads) {
            unsigned long long hits = 0;
            if (look) {
#pragma unroll 2
                for (int j = 0; j < 64 / V; ++j) {
                    const int q = q0 + j * kThreads + tid;
                    if (q >= packs) break;
                    const Pack<T> v = packed[q];
                    uint32_t m = 0;
#pragma unroll
                    for (int i = 0; i < V; ++i) m |= wanted(to_f32(v.e[i])) ? 1u << i : 0u;
                    hits |= static_cast<unsigned long long>(m) << (j * V);
                }
            }
            const int mine = __popcll(hits);
            if (!__any_sync(0xffffffffu, mine)) continue;
            int upto = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += y;
            }
            uint32_t base = 0;
            if (lane == 31) base = atomicAdd(&sh->n_mine, uint32_t(upto));
            uint32_t at = __shfl_sync(0xffffffffu, base, 31) + uint32_t(upto - mine);
            for (; hits && at < kList; hits &= hits - 1, ++at) {
                const int b = __ffsll(static_cast<long long>(hits)) - 1, e = (q0 + b / V * kThreads + tid) * V + b % V - shift;
                sh->cum[at] = uint64_t(order_key(to_f32(x[e]))) << 32 | uint32_t(~(first + e));
            }
        }
        __syncthreads();
        const uint32_t count = sh->n_mine;
        if (tid == 0 && count) sh->base = atomicAdd(&lead->n_list, count);
        __syncthreads();
        for (uint32_t i = tid; i < min(count, uint32_t(kList)) && sh->base + i < kList; i += kThreads)
            lead->list[sh->base + i] = sh->cum[i];
        if (tid == 0) sh->n_mine = 0;
        cluster_sync();
    };

    // (after a cluster barrier) The first CTA's bins[0, count) become the sums over all CTAs'.  Each CTA takes some that follow one
    // another: every eighth of them took eight times as long.
    auto sum_bins = [&](uint32_t *bins, int count) {
        const int some = count / cluster;  // (a multiple of 4)
        for (int b = int(rank) * some + 4 * tid; b < int(rank + 1) * some; b += 4 * kThreads) {
            uint4 c = make_uint4(0, 0, 0, 0);
#pragma unroll 4
            for (int o = 0; o < cluster; ++o) {
                const uint4 v = *reinterpret_cast<const uint4 *>(at_cta(bins, uint32_t(o)) + b);
                c = make_uint4(c.x + v.x, c.y + v.y, c.z + v.z, c.w + v.w);
            }
            *reinterpret_cast<uint4 *>(at_cta(bins, 0) + b) = c;
        }
        cluster_sync();
    };

    // ---- the head
    const bool all = a.vocab <= kList, guess = !all && !cut_k && !rw.only && rw.s_hi > 0.f;
    const bool try_head = all || rw.only || (cut_k && k <= kMostHeadK);
    if (try_head) {
        if (!all) {
            // maxima of groups of four threads, or, for many, of each
            const int want = cut_k ? k : 1;
            float m = mine;
            const bool fours = want <= kThreads / 8 || (want <= kRankSort && cluster == kMaxCluster);
            if (fours) {
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
            }
            const int b = !fours || (lane & 3) == 0 ? bin_of_logit(m) : -1;
            if (b >= 0) atomicAdd(&lead->count[b], 1u);
            cluster_sync();
            if (rank == 0) {
                constexpr int per = (kBins + kThreads - 1) / kThreads;
                uint32_t c[per], sum = 0;
#pragma unroll
                for (int j = 0; j < per; ++j) {
                    c[j] = tid * per + j < kBins ? sh->count[tid * per + j] : 0;
                    sum += c[j];
                }
                if (tid == 0) sh->found = kBins;
                uint32_t before = uint32_t(block_scan(sum, sh)) - sum;
#pragma unroll
                for (int j = 0; j < per; ++j) {
                    if (before < uint32_t(want) && before + c[j] >= uint32_t(want)) sh->found = tid * per + j;
                    before += c[j];
                }
                __syncthreads();
                // (none found: whatever has a weight)
                const float limit = sh->found == kBins ? float(kWeightBits + 1) : float(sh->found + 1) / per_unit;
                if (tid < cluster) at_cta(sh, uint32_t(tid))->floor = rw.floor_of(limit);
            }
            cluster_sync();
        }
        const float floor = all ? -3.402823466e38f : sh->floor;
        // (only of the packs that this thread brought, if any is there)
        collect(mine >= floor, [&](float v) { return v >= floor; });
    }

    // (first CTA) Sorts the list's `count` elements: this thread's weights and their cumulative ones, from `before` on (in
    // sh->cum too).
    unsigned long long w[kEach], cum[kEach];
    auto sort_and_sum = [&](int count, unsigned long long before) {
        sort_list(sh->list, sh->cum, count);
        unsigned long long sum = 0;
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
            const int i = tid * kEach + j;
            w[j] = i < count ? rw.weight(key_value(uint32_t(sh->list[i] >> 32)), sh->table) : 0;
            sum += w[j];
        }
        unsigned long long c = before + block_scan(sum, sh) - sum;
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
            c += w[j];
            cum[j] = c;
            sh->cum[tid * kEach + j] = c;
        }
        __syncthreads();
    };
    // (first CTA) The first of the `count` sorted elements whose cumulative weight is `mass` or more; `count`: none.
    auto first_of_mass = [&](unsigned long long mass, int count) {
        int below = 0;
#pragma unroll
        for (int j = 0; j < kEach; ++j) below += __syncthreads_count(tid * kEach + j < count && cum[j] < mass);
        return below;
    };
    auto write = [&](uint32_t index, uint64_t weight, unsigned long long kept) {
        a.tokens[r] = int64_t(index);
        if (a.prob) a.prob[r] = float(double(weight) / double(kept));
    };
    if (try_head) {
        if (rank == 0) {
            const int count = int(sh->n_list);
            const bool ok = count <= kList;
            if (ok) {  // (all that is kept is there)
                sort_and_sum(count, 0);
                unsigned long long kept = sh->cum[(cut_k ? min(k, count) : count) - 1];
                if (cut_p) kept = sh->cum[first_of_mass(mass_needed(p, kept), count)];
                if (least > 1) {
                    int heavy = 0;  // those that min_p keeps
#pragma unroll
                    for (int j = 0; j < kEach; ++j) heavy += __syncthreads_count(w[j] >= least);
                    kept = min(kept, sh->cum[heavy - 1]);
                }
                const int f = first_of_mass(drawn_mass(u, kept) + 1, count);
                if (tid == 0) write(~uint32_t(sh->list[f]), sh->cum[f] - (f ? sh->cum[f - 1] : 0), kept);
            }
            if (tid < cluster) at_cta(sh, uint32_t(tid))->cmd.op = ok ? OP_DONE : OP_HISTOGRAM;
        }
        cluster_sync();
        if (sh->cmd.op == OP_DONE) return;
    }

    // ---- a guess
    if (guess) {
        const float fine_per_unit = 4.f * per_unit;
        each([&](float v) {
            const float y = rw.coarse(v);
            if (y < float(kWeightBits + 1)) atomicAdd(&fine[min(int(y * fine_per_unit), kFine - 1)], 1u);
        });
        cluster_sync();
        sum_bins(fine, kFine);
        if (rank == 0) {
            // Cumulative weights of the bins, as if all their elements lay in the middle.  (Scanned in 2^-26, with the counts from
            // bit 45 on.)
            constexpr int per = (kFine + kThreads - 1) / kThreads;
            constexpr unsigned long long mask = (1ull << 45) - 1;
            const float unit = 1.f / fine_per_unit;
            auto of_bin = [&](int b) { return float(fine[b]) * exp2f(26.f - (float(b) + 0.5f) * unit); };
            const int b0 = min(tid * per, kFine), b1 = min(b0 + per, kFine);
            float weight = 0.f;
            uint32_t count = 0;
            for (int b = b0; b < b1; ++b) {
                weight += of_bin(b);
                count += fine[b];
            }
            const unsigned long long mine = static_cast<unsigned long long>(count) << 45 | static_cast<unsigned long long>(weight);
            const unsigned long long upto = block_scan(mine, sh), whole = sh->part[kWarps - 1];
            const float row = float(whole & mask), first = float((upto - mine) & mask), last = float(upto & mask);
            const uint32_t before = uint32_t((upto - mine) >> 45);
            if (tid < 4) {
                sh->edge[tid] = kFine;
                sh->until[tid] = uint32_t(whole >> 45);
            }
            if (tid < 2) sh->heavy[tid] = row;
            __syncthreads();
            // Edge i: the bin in which the cumulative weight passes `at`.
            auto find_edge = [&](int i, float at) {
                if (tid == 0 && !(at >= 0.f)) {
                    sh->edge[i] = 0;
                    sh->until[i] = 0;
                }
                if (!(first > at) && last > at) {
                    float c = first;
                    uint32_t n = before;
                    int b = b0;
                    for (; b < b1 - 1 && !((c += of_bin(b)) > at); ++b) n += fine[b];
                    sh->edge[i] = b + (i & 1);  // (whole bins: elements may be few, or lie on a grid as coarse as the bins)
                    sh->until[i] = n + (i & 1 ? fine[b] : 0);
                }
            };
            if (least > 1) {
                const int b = min(int((float(kWeightBits) - log2f(float(least))) * fine_per_unit), kFine - 1);
                if (b >= b0 && b < b1) {
                    float c = first;
                    for (int j = b0; j < b; ++j) c += of_bin(j);
                    sh->heavy[0] = c;
                    sh->heavy[1] = c + of_bin(b);
                }
            }
            // three times what the places of elements within their bins may add up to (their standard deviation, with the sum of
            // squared weights at most the sum), twice that where what is kept is a guess too
            const float slack = 0.6f * unit * sqrtf(row * 0x1p26f);
            const float target = cut_p ? row * fmaxf(p, 0.f) : row;
            if (cut_p) {
                find_edge(0, target - slack);
                find_edge(1, target + slack);
            }
            __syncthreads();
            // (top_p keeps the element that it ends in, and so up to the weight of one at its range's upper end more)
            const float over = cut_p ? exp2f(26.f - float(sh->edge[0]) * unit) : 0.f, part = fminf(fmaxf(u, 0.f), 1.f);
            find_edge(2, part * fminf(target, sh->heavy[0]) - 2.f * slack);
            find_edge(3, part * fminf(target + over, sh->heavy[1]) + 2.f * slack);
            __syncthreads();
            if (tid < cluster) {
                Shared *to = at_cta(sh, uint32_t(tid));
                to->found = (cut_p ? sh->until[1] - sh->until[0] : 0) + sh->until[3] - sh->until[2] <= kList;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const bool off = i == 0 && !cut_p;
                    to->range[i][0] = off ? INFINITY : rw.top - float(sh->edge[2 * i + 1]) * unit / rw.s_hi;
                    to->range[i][1] = off ? INFINITY : rw.top - float(sh->edge[2 * i]) * unit / rw.s_hi;
                }
            }
        }
        cluster_sync();
        if (sh->found) {
            const float lo1 = sh->range[0][0], hi1 = sh->range[0][1], lo2 = sh->range[1][0], hi2 = sh->range[1][1];
            unsigned long long sums[4] = {};
            for (int q = tid; q < packs; q += kThreads) {
                const Pack<T> v = packed[q];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float f = to_f32(v.e[i]);
                    const unsigned long long w = rw.weight(f, sh->table);
                    sums[0] += w;
                    sums[1] += w >= least ? w : 0;
                    sums[2] += f > hi1 ? w : 0;
                    sums[3] += f > hi2 ? w : 0;
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
#pragma unroll
                for (int o = 16; o; o >>= 1) sums[j] += __shfl_xor_sync(0xffffffffu, sums[j], o);
                if (lane == 0 && sums[j]) atomicAdd(&sh->my_sums[j], sums[j]);
            }
            __syncthreads();
            if (tid < 4) atomicAdd(&lead->sums[tid], sh->my_sums[tid]);
            collect(true, [&](float v) { return ((v >= lo1) & (v <= hi1)) | ((v >= lo2) & (v <= hi2)); });
        }
        if (rank == 0) {
            const int count = int(sh->n_list);
            bool ok = sh->found && count > 0 && count <= kList;
            if (ok) {
                sort_and_sum(count, 0);
                // The list's element at which the prefix reaches `target`, if it lies in range i; *skip: what is to be added to
                // the list's cumulative weights there.
                auto find = [&](unsigned long long target, int i, unsigned long long *skip) {
                    const float lo = sh->range[i][0], hi = sh->range[i][1];
                    int from = 0, to = 0;
#pragma unroll
                    for (int j = 0; j < kEach; ++j) {
                        const int e = tid * kEach + j;
                        const float v = e < count ? key_value(uint32_t(sh->list[e] >> 32)) : -INFINITY;
                        from += __syncthreads_count(v > hi);
                        to += __syncthreads_count(v >= lo);
                    }
                    const unsigned long long above = sh->sums[2 + i], before = from ? sh->cum[from - 1] : 0;
                    *skip = above - before;  // (modulo 2^64)
                    if (target <= above) return -1;
                    const int f = first_of_mass(target - *skip, count);
                    return f < to ? f : -1;
                };
                unsigned long long kept = sh->sums[0], skip;
                if (cut_p) {
                    const int f = find(mass_needed(p, kept), 0, &skip);
                    ok = f >= 0;
                    if (ok) kept = sh->cum[f] + skip;
                }
                if (least > 1) kept = min(kept, sh->sums[1]);
                const int f = ok ? find(drawn_mass(u, kept) + 1, 1, &skip) : -1;
                ok = f >= 0;
                if (ok && tid == 0) write(~uint32_t(sh->list[f]), sh->cum[f] - (f ? sh->cum[f - 1] : 0), kept);
            }
            if (tid < cluster) at_cta(sh, uint32_t(tid))->cmd.op = ok ? OP_DONE : OP_HISTOGRAM;
        }
        cluster_sync();
        if (sh->cmd.op == OP_DONE) return;
    }

    // ---- the whole order
    // Counts and weights of the bins slot(x) of all CTAs' elements (below 0: none), in the first CTA.
    auto histogram = [&](auto slot) {
        for (int i = tid; i < kBins; i += kThreads) sh->count[i] = sh->mass[0][i] = sh->mass[1][i] = sh->mass[2][i] = 0;
        __syncthreads();
        for (int q = tid; q < packs; q += kThreads) {
            const Pack<T> v = packed[q];
#pragma unroll
            for (int i0 = 0; i0 < V; i0 += 4) {
                int b[4];
                uint64_t w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    b[i] = slot(to_f32(v.e[i0 + i]));
                    w[i] = rw.weight(to_f32(v.e[i0 + i]), sh->table);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (b[i] >= 0) {
                        atomicAdd(&sh->count[b[i]], 1u);
                        atomicAdd(&sh->mass[0][b[i]], uint32_t(w[i]) & 0x7fffu);
                        atomicAdd(&sh->mass[1][b[i]], uint32_t(w[i] >> 15) & 0x7fffu);
                        atomicAdd(&sh->mass[2][b[i]], uint32_t(w[i] >> 30));
                    }
            }
        }
        cluster_sync();
        const int some = kBins / cluster;
        for (int b = int(rank) * some + tid; b < int(rank + 1) * some; b += kThreads) {
            uint32_t c = 0;
            unsigned long long m = 0;
            for (int o = 0; o < cluster; ++o) {
                const Shared *from = at_cta(sh, uint32_t(o));
                c += from->count[b];
                m += from->mass[0][b] + (uint64_t(from->mass[1][b]) << 15) + (uint64_t(from->mass[2][b]) << 30);
            }
            lead->count[b] = c;
            lead->mass[0][b] = uint32_t(m);
            lead->mass[1][b] = uint32_t(m >> 32);
        }
        cluster_sync();
    };
    auto mass_of = [&](int b) { return sh->mass[0][b] | static_cast<unsigned long long>(sh->mass[1][b]) << 32; };
    // Has every CTA do `c` (first CTA: all its threads call it), up to the results' being there.
    auto work = [&](const Command &c) {
        if (c.op == OP_HISTOGRAM) {
            histogram([&](float v) { return bin_of_logit(v); });
        } else if (c.op == OP_REFINE) {
            histogram([&](float v) {
                const uint32_t key = order_key(v);
                return (key >= c.low) & (key <= c.high) & (bin_of_logit(v) == c.bin) ? int((c.high - key) >> c.shift) : -1;
            });
        } else if (c.op == OP_SPAN) {  // the smallest and largest key of a bin
            uint32_t lo = 0xffffffffu, hi = 0;
            each([&](float v) {
                const bool in = bin_of_logit(v) == c.bin;
                lo = min(lo, in ? order_key(v) : 0xffffffffu);
                hi = max(hi, in ? order_key(v) : 0u);
            });
            lo = __reduce_min_sync(0xffffffffu, lo);
            hi = __reduce_max_sync(0xffffffffu, hi);
            if (lane == 0 && lo <= hi) {
                atomicMin(&lead->low, lo);
                atomicMax(&lead->high, hi);
            }
            cluster_sync();
        } else if (c.op == OP_GATHER) {
            collect(true, [&](float v) {
                const uint32_t key = order_key(v);
                return (key >= c.low) & (key <= c.high) & (bin_of_logit(v) == c.bin);
            });
        } else if (c.op == OP_HEAVY) {  // the weight of what min_p keeps
            unsigned long long sum = 0;
            each([&](float v) {
                const uint64_t w = rw.weight(v, sh->table);
                sum += w >= least ? w : 0;
            });
#pragma unroll
            for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (lane == 0 && sum) atomicAdd(&lead->total, sum);
            cluster_sync();
        } else if (c.op == OP_TIE) {  // the CTA that holds the wanted one of the equal elements writes it
            uint32_t same = 0;
            const int per = (slice + kThreads - 1) / kThreads, i0 = tid * per, i1 = min(n, i0 + per);
            for (int i = i0; i < i1; ++i) same += order_key(to_f32(x[i])) == c.low;
            const uint32_t upto = uint32_t(block_scan(same, sh));
            if (tid == kThreads - 1)
                for (int o = 0; o < cluster; ++o) at_cta(sh, uint32_t(o))->ties[rank] = upto;
            cluster_sync();
            uint32_t before = upto - same;
            for (int o = 0; o < int(rank); ++o) before += sh->ties[o];
            for (int i = i0; i < i1; ++i)
                if (order_key(to_f32(x[i])) == c.low && before++ == c.rank)
                    write(uint32_t(first + i), rw.weight(to_f32(x[i]), sh->table), lead->kept);
            cluster_sync();
        }
    };
    if (rank != 0) {
        for (;;) {
            cluster_sync();
            const Command c = sh->cmd;
            if (c.op == OP_DONE) return;
            work(c);
        }
    }
    auto command = [&](const Command &c) {
        if (tid < cluster) at_cta(sh, uint32_t(tid))->cmd = c;
        cluster_sync();
        if (c.op != OP_DONE) work(c);
        __syncthreads();
    };
    bool fresh = false;  // the bins' histogram stands
    struct Place {
        unsigned long long before, mass;  // weight before the element, and up to it
        uint32_t index;
        bool tie;  // index: which of the elements `key`
        uint32_t key;
    };
    // The first bin of the histogram in which the prefix reaches `target` (a count or a weight); what lies before it.
    auto bin_of = [&](bool by_count, unsigned long long target, int bins, unsigned long long base_count,
                      unsigned long long base_mass, unsigned long long *count, unsigned long long *mass) {
        constexpr int per = (kBins + kThreads - 1) / kThreads;
        unsigned long long c = 0, m = 0;
        for (int j = 0; j < per; ++j) {
            const int b = tid * per + j;
            if (b < bins) {
                c += sh->count[b];
                m += mass_of(b);
            }
        }
        unsigned long long c0 = base_count + block_scan(c, sh) - c;
        unsigned long long m0 = base_mass + block_scan(m, sh) - m;
        if (tid == 0) sh->found = -1;
        __syncthreads();
        for (int j = 0; j < per; ++j) {
            const int b = tid * per + j;
            if (b >= bins) break;
            const unsigned long long c1 = c0 + sh->count[b], m1 = m0 + mass_of(b);
            if (by_count ? c0 < target && c1 >= target : m0 < target && m1 >= target) {
                sh->found = b;
                sh->found_before = c0;
                sh->found_mass = m0;
            }
            c0 = c1;
            m0 = m1;
        }
        __syncthreads();
        const int f = sh->found;
        *count = sh->found_before;
        *mass = sh->found_mass;
        __syncthreads();
        return f;
    };
    // The first element of the order whose prefix reaches `target`.
    auto place_of = [&](bool by_count, unsigned long long target) {
        if (!fresh) command(Command{OP_HISTOGRAM});
        fresh = true;
        unsigned long long count, mass;
        const int bin = bin_of(by_count, target, kBins, 0, 0, &count, &mass);
        uint32_t in = sh->count[bin], low = 0, high = 0xffffffffu;
        if (in > kList) {
            if (tid == 0) {
                sh->low = 0xffffffffu;
                sh->high = 0;
            }
            __syncthreads();
            command(Command{OP_SPAN, bin});
            low = sh->low;
            high = sh->high;
            while (in > kList && low < high) {
                int shift = 0;
                while ((high - low) >> shift >= kBins) ++shift;
                command(Command{OP_REFINE, bin, shift, low, high});
                fresh = false;
                const int sub = bin_of(by_count, target, kBins, count, mass, &count, &mass);
                in = sh->count[sub];
                __syncthreads();
                high -= uint32_t(sub) << shift;
                low = max(low, high - ((1u << shift) - 1));
            }
        }
        Place at = {};
        if (in > kList) {  // equal elements
            const uint64_t w = rw.weight(key_value(low), sh->table);
            const unsigned long long which = by_count ? target - count - 1 : (target - mass - 1) / w;
            at.tie = true;
            at.key = low;
            at.index = uint32_t(which);
            at.before = mass + which * w;
            at.mass = at.before + w;
            return at;
        }
        if (tid == 0) sh->n_list = 0;
        __syncthreads();
        command(Command{OP_GATHER, bin, 0, low, high});
        sort_and_sum(int(in), mass);
        const int f = by_count ? int(target - count) - 1 : first_of_mass(target, int(in));
        at.mass = sh->cum[f];
        at.before = f ? sh->cum[f - 1] : mass;
        at.index = ~uint32_t(sh->list[f]);
        __syncthreads();
        return at;
    };
    command(Command{OP_HISTOGRAM});
    fresh = true;
    unsigned long long kept;
    uint32_t there;
    {
        unsigned long long c = 0, m = 0;
        for (int b = tid; b < kBins; b += kThreads) {
            c += sh->count[b];
            m += mass_of(b);
        }
        c = block_scan(c, sh);
        if (tid == kThreads - 1) sh->found_before = c;
        m = block_scan(m, sh);
        if (tid == kThreads - 1) sh->found_mass = m;
        __syncthreads();
        there = uint32_t(sh->found_before);
        kept = sh->found_mass;
        __syncthreads();
    }
    if (cut_k && uint32_t(k) < there) kept = place_of(true, unsigned(k)).mass;
    if (cut_p) kept = place_of(false, mass_needed(p, kept)).mass;
    if (least > 1) {
        if (tid == 0) sh->total = 0;
        __syncthreads();
        command(Command{OP_HEAVY});
        kept = min(kept, sh->total);
    }
    const Place at = place_of(false, drawn_mass(u, kept) + 1);
    if (at.tie) {
        if (tid == 0) sh->kept = kept;
        __syncthreads();
        command(Command{OP_TIE, 0, 0, at.key, at.key, at.index});
    } else if (tid == 0) {
        write(at.index, at.mass - at.before, kept);
    }
    command(Command{OP_DONE});
}

// Shared memory of a CTA that holds `slice` logits: at most those of the largest vocabulary over the most CTAs, as more CTAs take
// a row as long as a slice has more than 64 KB.
template <typename T>
constexpr size_t shared_bytes(int slice) {
    return sizeof(Shared) + size_t(slice) * sizeof(T) + 32;
}
static_assert(kMaxVocab / kMaxCluster * 2 >= 65536 && shared_bytes<float>(kMaxVocab / kMaxCluster) <= 232448);

template <typename T>
cudaError_t launch(const SampleArgs &a, const LaunchCtx &ctx) {
    // CTAs of a row: at least as many as its slices need to let two CTAs share an SM, more where rows are few
    int cluster = 1;
    while (cluster < kMaxCluster && int64_t(a.vocab) * int64_t(sizeof(T)) > int64_t(cluster) * 65536) cluster *= 2;
    while (cluster < kMaxCluster && a.rows * cluster * 2 <= 2 * ctx.num_sms && a.vocab > cluster * 2048) cluster *= 2;
    const int slice = ((a.vocab + cluster - 1) / cluster + 7) & ~7;
    const size_t smem = shared_bytes<T>(slice);
    auto kernel = sample_kernel<T>;
    // (the process's, so that calls of several threads all ask for the same: a smaller one could come between another's and its
    // launch)
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(shared_bytes<T>(kMaxVocab / kMaxCluster)));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(a.rows * cluster));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
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
    return cudaLaunchKernelEx(&cfg, kernel, a, slice, cluster);
}

}  // namespace

cudaError_t launch_sample(const SampleArgs &a, int dtype, const LaunchCtx &ctx) {
    switch (dtype) {
        case TQ2_F32: return launch<float>(a, ctx);
        case TQ2_F16: return launch<__half>(a, ctx);
        default: return launch<__nv_bfloat16>(a, ctx);
    }
}

}  // namespace tq2
