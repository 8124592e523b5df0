// Routing: the top_k experts of each token by its logits, and their weights.
//
// Order: logits descending, equal ones by index, NaN last; softmax and sigmoid do not change it, so the choice
// is one of exact comparisons and no rounding decides it.  The weights are scores over the logits (softmax over all
// experts, or a sigmoid each), divided by their sum over the chosen where asked.
//
// A warp takes a token: each lane holds NV logits as integers in the order of their values.  Of 16-bit logits the index
// fits below the value in one word, all different: a lane sorts its own by a network once, and top_k times the warp's largest
// head (one redux) leaves its lane's list.  Of f32 ones: top_k times the warp's maximum, the lowest index that holds it
// (another redux), and each lane's maximum anew.
//
// Bound by issue slots and the loads' latency: 8 of 256 bf16 logits of 8191 tokens (4.2 MB read) take 6.5 us, 485 warp
// instructions a token, half of the issue slots (without the sorted lists, as f32 ones are chosen: 10.4 us, 793; 32 of 1024:
// 35 against 83 us); one token 1.9 us, its launch.  Calls from Python take 13 us (two new tensors, the checks and the launch).
#include <cstdint>
#include <type_traits>

#include "dtype.cuh"
#include "tq2_internal.cuh"

namespace tq2 {
namespace {

constexpr int kWarps = 8;  // tokens of a block

// Descending, by Batcher's merging network: sorted runs of P, from places D apart on.
template <int N, int P = 1, int D = 1>
__device__ __forceinline__ void sort_lane(uint32_t (&k)[N]) {
#pragma unroll
    for (int i = D % P; i < N - D; ++i)
        if ((i - D % P) / D % 2 == 0 && i / (2 * P) == (i + D) / (2 * P)) {
            const uint32_t high = max(k[i], k[i + D]), low = min(k[i], k[i + D]);
            k[i] = high;
            k[i + D] = low;
        }
    if constexpr (D > 1)
        sort_lane<N, P, D / 2>(k);
    else if constexpr (2 * P < N)
        sort_lane<N, 2 * P, 2 * P>(k);
}

template <typename T, int NV>
__global__ void __launch_bounds__(32 * kWarps)
moe_route_kernel(const T *__restrict__ logits, int64_t row_stride, int32_t *__restrict__ experts,
                 float *__restrict__ weights, int64_t tokens, int n, int top_k, int sigmoid, int normalize, float scale) {
    const int lane = threadIdx.x & 31;
    const int64_t t = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (t >= tokens) return;
    const T *row = logits + t * row_stride;
    // 16-bit logits: what an f32 of theirs never uses, in which the index stands (from above)
    constexpr bool WORD = sizeof(T) == 2;
    constexpr uint32_t LOW = std::is_same_v<T, __half> ? 0x1fffu : 0xffffu;
    auto value_of = [](uint32_t k) {
        if (!WORD) return key_value(k);
        const uint32_t v = k & ~LOW;
        return key_value(v == 0 ? 1u : (v & 0x80000000u) ? v : v | LOW);
    };
    uint32_t key[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int i = j * 32 + lane;
        key[j] = i < n ? order_key(to_f32(row[i])) : 0u;  // 0: none, or taken
        if (WORD && i < n) key[j] = (key[j] & ~LOW) | (LOW - uint32_t(i));
    }
    uint32_t best = 0;
    bool nan = false;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        best = max(best, key[j]);
        nan |= WORD ? key[j] - 1u < LOW : key[j] == order_key(__uint_as_float(0x7fc00000u));
    }
    nan = __any_sync(0xffffffffu, nan);
    const float top = value_of(__reduce_max_sync(0xffffffffu, best));
    float z = 1.f;  // the softmax's denominator
    if (!sigmoid && !normalize) {
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (key[j]) s += expf(value_of(key[j]) - top);
#pragma unroll
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        z = s;
    }
    int mine = 0;            // lane j: the j-th expert and its logit
    float value = 0.f;
    if constexpr (WORD) {
        sort_lane(key);
        uint32_t taken = 1;
        for (int k = 0; k < top_k; ++k) {
            const uint32_t m = __reduce_max_sync(0xffffffffu, key[0]);
            const bool own = key[0] == m;
#pragma unroll
            for (int j = 0; j + 1 < NV; ++j) key[j] = own ? key[j + 1] : key[j];
            key[NV - 1] = own ? 0u : key[NV - 1];
            taken = lane == k ? m : taken;
        }
        mine = int(LOW - (taken & LOW));
        value = value_of(taken);
    } else {
        for (int k = 0; k < top_k; ++k) {
            const uint32_t m = __reduce_max_sync(0xffffffffu, best);
            int at = INT32_MAX;
            if (best == m) {
#pragma unroll
                for (int j = NV - 1; j >= 0; --j)
                    if (key[j] == m) at = j * 32 + lane;
            }
            const int i = __reduce_min_sync(0xffffffffu, at);
            if (at == i) {
                best = 0;
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    if (j * 32 + lane == i) key[j] = 0u;
                    best = max(best, key[j]);
                }
            }
            if (lane == k) {
                mine = i;
                value = key_value(m);
            }
        }
    }
    float s = 0.f;
    if (lane < top_k && value != -INFINITY) {
        if (!sigmoid) {
            s = expf(value - top);
        } else if (!(value < 0.f)) {
            s = 1.f / (1.f + expf(-value));
        } else {  // (normalised, times exp(-top) where that is below 0 too: sigmoids that underflow have quotients all the same)
            s = expf(normalize ? value - fminf(top, 0.f) : value) / (1.f + expf(value));
        }
    }
    float sum = z;
    if (normalize) {
        sum = s;
#pragma unroll
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    if (lane < top_k) {
        experts[t * top_k + lane] = mine;
        float w = s == 0.f && !(sum != sum) ? 0.f : (sigmoid && !normalize ? s : s / sum) * scale;
        if (top == -INFINITY && !nan) w = 0.f;                            // nothing but -inf
        if (!sigmoid && (nan || top == INFINITY)) w = __uint_as_float(0x7fc00000u);  // (in the softmax's sum, chosen or not)
        weights[t * top_k + lane] = w;
    }
}

template <typename T>
cudaError_t launch(const RouteArgs &a, const LaunchCtx &ctx) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned((a.tokens + kWarps - 1) / kWarps));
    cfg.blockDim = dim3(32 * kWarps);
    cfg.stream = ctx.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    auto go = [&](auto kern) {
        return cudaLaunchKernelEx(&cfg, kern, static_cast<const T *>(a.logits), a.row_stride, a.experts, a.weights,
                                  a.tokens, a.n, a.top_k, a.sigmoid, a.normalize, a.scale);
    };
    if (a.n <= 64) return go(moe_route_kernel<T, 2>);
    if (a.n <= 128) return go(moe_route_kernel<T, 4>);
    if (a.n <= 256) return go(moe_route_kernel<T, 8>);
    if (a.n <= 512) return go(moe_route_kernel<T, 16>);
    return go(moe_route_kernel<T, 32>);
}

}  // namespace

cudaError_t launch_moe_route(const RouteArgs &a, int dtype, const LaunchCtx &ctx) {
    switch (dtype) {
        case TQ2_F32: return launch<float>(a, ctx);
        case TQ2_F16: return launch<__half>(a, ctx);
        default: return launch<__nv_bfloat16>(a, ctx);
    }
}

}  // namespace tq2
