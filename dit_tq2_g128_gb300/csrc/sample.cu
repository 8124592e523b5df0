// Sampling: one token of each row of logits, by a given random number.
//
// Tokens are ordered by their logits, descending, equal ones by index.  Weights w = exp((l - max) / temperature) are
// integers in units of 2^-45, so that sums of them are exact in any order; temperature, top-k, top-p and min-p each keep
// a prefix of the order, and the token drawn is the first whose cumulative weight passes u times the kept weight.
// Every question is then one of counts or sums over a prefix.
//
// The plain form: a block a row, each question by bisection over the order's integers.
#include <cstdint>

#include "dtype.cuh"
#include "sample_weight.cuh"
#include "tq2_internal.cuh"

namespace tq2 {
namespace {

constexpr int kThreads = 1024;

struct Sum {
    uint64_t count, mass;
};

__device__ Sum block_sum(Sum v, Sum *part) {
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        v.count += __shfl_xor_sync(0xffffffffu, v.count, o);
        v.mass += __shfl_xor_sync(0xffffffffu, v.mass, o);
    }
    __syncthreads();
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    Sum s = {0, 0};
    for (int w = 0; w < kThreads / 32; ++w) {
        s.count += part[w].count;
        s.mass += part[w].mass;
    }
    return s;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) sample_kernel(SampleArgs a) {
    __shared__ Sum part[kThreads / 32];
    __shared__ uint64_t table[64];
    __shared__ uint32_t highest[kThreads / 32];
    const int64_t r = blockIdx.x;
    const T *row = static_cast<const T *>(a.logits) + r * a.row_stride;
    fill_weight_table(table);
    uint32_t best = 0;
    for (int i = threadIdx.x; i < a.vocab; i += kThreads) best = max(best, order_key(to_f32(row[i])));
    best = __reduce_max_sync(0xffffffffu, best);
    if ((threadIdx.x & 31) == 0) highest[threadIdx.x >> 5] = best;
    __syncthreads();
    for (int w = 0; w < kThreads / 32; ++w) best = max(best, highest[w]);
    const RowWeights rw(key_value(best), a.temperature ? a.temperature[r] : 1.f);
    auto place = [&](int i) { return uint64_t(order_key(to_f32(row[i]))) << 18 | uint64_t(kMaxVocab - 1 - i); };
    // of the prefix of the tokens whose place is `from` or more
    auto prefix = [&](uint64_t from, uint64_t least) {
        Sum s = {0, 0};
        for (int i = threadIdx.x; i < a.vocab; i += kThreads)
            if (place(i) >= from) {
                const uint64_t w = rw.weight(to_f32(row[i]), table);
                s.mass += w >= least ? w : 0;
                ++s.count;
            }
        return block_sum(s, part);
    };
    // the last place whose prefix fulfils `enough`
    auto find = [&](auto enough) {
        uint64_t lo = 0, hi = uint64_t(1) << 50;  // enough at lo, not at hi
        while (hi - lo > 1) {
            const uint64_t mid = (lo + hi) / 2;
            if (enough(prefix(mid, 0))) lo = mid;
            else hi = mid;
        }
        return lo;
    };
    if (best <= order_key(-INFINITY)) {
        if (threadIdx.x == 0) {
            a.tokens[r] = -1;
            if (a.prob) a.prob[r] = 0.f;
        }
        return;
    }
    uint64_t kept = prefix(0, 0).mass;
    const int k = a.top_k ? a.top_k[r] : 0;
    if (k > 0 && k < a.vocab) kept = prefix(find([&](Sum s) { return s.count >= uint64_t(k); }), 0).mass;
    if (a.top_p && a.top_p[r] < 1.f) {
        const uint64_t need = mass_needed(a.top_p[r], kept);
        kept = prefix(find([&](Sum s) { return s.mass >= need; }), 0).mass;
    }
    if (a.min_p) kept = min(kept, prefix(0, least_weight(a.min_p[r])).mass);
    const uint64_t passed = drawn_mass(a.u[r], kept);
    const uint64_t at = find([&](Sum s) { return s.mass > passed; });
    if (threadIdx.x == 0) {
        const int i = kMaxVocab - 1 - int(at & (kMaxVocab - 1));
        a.tokens[r] = i;
        if (a.prob) a.prob[r] = float(double(rw.weight(to_f32(row[i]), table)) / double(kept));
    }
}

}  // namespace

cudaError_t launch_sample(const SampleArgs &a, int dtype, const LaunchCtx &ctx) {
    const dim3 grid(static_cast<unsigned>(a.rows));
    switch (dtype) {
        case TQ2_F32: sample_kernel<float><<<grid, kThreads, 0, ctx.stream>>>(a); break;
        case TQ2_F16: sample_kernel<__half><<<grid, kThreads, 0, ctx.stream>>>(a); break;
        default: sample_kernel<__nv_bfloat16><<<grid, kThreads, 0, ctx.stream>>>(a); break;
    }
    return cudaGetLastError();
}

}  // namespace tq2
