// Mixture of ternary experts:
//     out[t] = residual[t] + sum_j weight[t, j] Down_e (silu(Gate_e x_t) * (Up_e x_t)),  e = expert[t, j].
//
// The plain form: a warp for each feature of each (token, expert) pair, then one for each element of the output.
#include <cstdint>

#include "dtype.cuh"
#include "tq2_internal.cuh"

namespace tq2 {
namespace {

// Lane's part of the product of row `row` of a ternary weight with v.
template <typename V>
__device__ __forceinline__ float dot_part(const SoaView &w, int64_t row, int blocks, const V *v, int lane) {
    float acc = 0.f;
    for (int b = 0; b < blocks; ++b) {
        const uint32_t q = w.qs[(row * blocks + b) * kQsBytes + lane];
        const float d = __half2float(w.d[row * blocks + b]);
        const V *x = v + b * kBlockW + 4 * lane;
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) s = fmaf(float(int(q >> 2 * j & 3) - 1), to_f32(x[j]), s);
        acc = fmaf(d, s, acc);
    }
    return acc;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

template <typename T>
__global__ void __launch_bounds__(256) moe_hidden_kernel(MoeArgs a, SoaView w, float *__restrict__ h, unsigned int *status) {
    const int lane = threadIdx.x & 31;
    const int64_t items = a.tokens * a.top_k * a.ffn, step = int64_t(gridDim.x) * 8;
    for (int64_t i = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5); i < items; i += step) {
        const int64_t p = i / a.ffn, f = i - p * a.ffn;
        const int e = a.expert[p];
        if (e < 0 || e >= a.experts) {
            if (f == 0 && lane == 0) report_bad(e != -1, status);
            continue;
        }
        const T *x = static_cast<const T *>(a.x) + p / a.top_k * a.width;
        const int64_t row = int64_t(e) * 2 * a.ffn + f;
        const float g = warp_sum(dot_part(w, row, a.width / kBlockW, x, lane));
        const float u = warp_sum(dot_part(w, row + a.ffn, a.width / kBlockW, x, lane));
        if (lane == 0) h[i] = g / (1.f + expf(-g)) * u;
    }
}

template <typename T>
__global__ void __launch_bounds__(256) moe_out_kernel(MoeArgs a, SoaView w, const float *__restrict__ h) {
    const int lane = threadIdx.x & 31;
    const int64_t items = a.tokens * a.width, step = int64_t(gridDim.x) * 8;
    for (int64_t i = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5); i < items; i += step) {
        const int64_t t = i / a.width, c = i - t * a.width;
        float sum = a.residual ? to_f32(static_cast<const T *>(a.residual)[i]) : 0.f;
        for (int64_t p = t * a.top_k; p < (t + 1) * a.top_k; ++p) {
            const int e = a.expert[p];
            if (e < 0 || e >= a.experts) continue;
            sum = fmaf(a.weight[p], warp_sum(dot_part(w, int64_t(e) * a.width + c, a.ffn / kBlockW, h + p * a.ffn, lane)),
                       sum);
        }
        __syncwarp();
        if (lane == 0) static_cast<T *>(a.out)[i] = from_f32<T>(sum);
    }
}

template <typename T>
cudaError_t launch(const MoeArgs &a, void *ws, const LaunchCtx &ctx) {
    float *h = static_cast<float *>(ws);
    moe_hidden_kernel<T><<<ctx.num_sms * 8, 256, 0, ctx.stream>>>(
        a, soa_view(a.gate_up, int64_t(a.experts) * 2 * a.ffn, a.width), h, ctx.status);
    moe_out_kernel<T><<<ctx.num_sms * 8, 256, 0, ctx.stream>>>(a, soa_view(a.down, int64_t(a.experts) * a.width, a.ffn), h);
    return cudaGetLastError();
}

}  // namespace

size_t moe_ws_bytes(int64_t tokens, int64_t top_k, int64_t experts, int64_t width, int64_t ffn, int dtype) {
    return size_t(tokens * top_k * ffn) * 4;
}

cudaError_t launch_moe(const MoeArgs &a, int dtype, void *ws, const LaunchCtx &ctx) {
    switch (dtype) {
        case TQ2_F32: return launch<float>(a, ws, ctx);
        case TQ2_F16: return launch<__half>(a, ws, ctx);
        default: return launch<__nv_bfloat16>(a, ws, ctx);
    }
}

}  // namespace tq2
