// Attention of a step's new tokens over a paged key/value cache.
//
// One warp per (token, head): lanes share the head's elements, keys one after the
// other with the running maximum and sum of the softmax, all in f32.
#include <cuda_bf16.h>

#include "tq2_internal.cuh"

namespace tq2 {
namespace {

constexpr int kWarps = 4;

__device__ __forceinline__ float up(__half x) { return __half2float(x); }
__device__ __forceinline__ float up(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float x, float *p) { *p = x; }
__device__ __forceinline__ void put(float x, __half *p) { *p = __float2half_rn(x); }
__device__ __forceinline__ void put(float x, __nv_bfloat16 *p) { *p = __float2bfloat16_rn(x); }

template <typename T, typename TO>
__global__ void __launch_bounds__(32 * kWarps) paged_row_kernel(const PagedArgs a, unsigned int *status) {
    const int lane = threadIdx.x & 31;
    const int64_t row = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const int64_t t = row / a.heads;
    const int h = int(row - t * a.heads);
    if (t >= a.batch.tokens) return;
    const int b = seq_of(a.batch, t);
    if (b < 0) return;
    bool bad = false;
    const SeqSpan sp = seq_span(a.batch, b, bad);
    if (t < sp.q0 || t >= int64_t(sp.q0) + sp.n) return;
    const KeyRange kr = keys_of(sp, int(t - sp.q0), a.window, a.causal);
    const T *q = static_cast<const T *>(a.q) + t * a.q_token + int64_t(h) * a.q_head;
    const int64_t head = int64_t(h / (a.heads / a.kv_heads)) * a.head_stride;
    float qr[4], o[4] = {0.f, 0.f, 0.f, 0.f}, m = -INFINITY, l = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) qr[i] = lane + 32 * i < a.dim ? up(q[lane + 32 * i]) : 0.f;
    for (int j = kr.lo; j < kr.hi; ++j) {
        const int in_table = j / a.batch.page_size;
        const int64_t page = page_of(a.batch, b, in_table, bad);
        if (page < 0) continue;
        const int64_t at = page * a.page_stride + int64_t(j - in_table * a.batch.page_size) * a.slot_stride + head;
        const T *k = static_cast<const T *>(a.k) + at, *v = static_cast<const T *>(a.v) + at;
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (lane + 32 * i < a.dim) s = fmaf(qr[i], up(k[lane + 32 * i]), s);
#pragma unroll
        for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
        s *= a.scale;
        const float mn = fmaxf(m, s);
        const float c = m == mn ? 1.f : expf(m - mn), p = s == mn ? 1.f : expf(s - mn);
        l = l * c + p;
        m = mn;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (lane + 32 * i < a.dim) o[i] = fmaf(p, up(v[lane + 32 * i]), o[i] * c);
    }
    TO *out = static_cast<TO *>(a.out) + t * a.out_token + int64_t(h) * a.out_head;
    const float inv = l > 0.f ? 1.f / l : (kr.hi > kr.lo ? l : 0.f);
    report_bad(bad, status);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (lane + 32 * i < a.dim) put(o[i] * inv, out + lane + 32 * i);
}

}  // namespace

cudaError_t launch_attention_paged_chunk(const PagedArgs &a, int dtype, bool out_f32, void *, const LaunchCtx &ctx) {
    const int64_t blocks = (a.batch.tokens * a.heads + kWarps - 1) / kWarps;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    const unsigned g = unsigned(blocks), n = 32 * kWarps;
    if (dtype == TQ2_F16) {
        if (out_f32) paged_row_kernel<__half, float><<<g, n, 0, ctx.stream>>>(a, ctx.status);
        else paged_row_kernel<__half, __half><<<g, n, 0, ctx.stream>>>(a, ctx.status);
    } else {
        if (out_f32) paged_row_kernel<__nv_bfloat16, float><<<g, n, 0, ctx.stream>>>(a, ctx.status);
        else paged_row_kernel<__nv_bfloat16, __nv_bfloat16><<<g, n, 0, ctx.stream>>>(a, ctx.status);
    }
    return cudaPeekAtLastError();
}

}  // namespace tq2
