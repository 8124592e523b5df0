// Loads and stores of the activation types as f32 (tq2_dtype).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace tq2 {

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// A float's place in the order of values, as an unsigned integer: equal zeros, NaN (either sign) below all.
__device__ __forceinline__ uint32_t order_key(float x) {
    if (x != x) return 1u;
    const uint32_t b = __float_as_uint(x + 0.0f);  // (-0 + 0 = +0)
    return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
    if (k == 1u) return __uint_as_float(0x7fc00000u);
    return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
}

}  // namespace tq2
