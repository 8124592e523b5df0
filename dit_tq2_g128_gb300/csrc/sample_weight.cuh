// The weight of a token in sampling, as an integer in units of 2^-45 of the likeliest token's.
//
// w = 2^-y, y = (max - l) log2(e) / temperature.  y is kept as a sum of two f32 (its error is 2^-46 of it), split into
// n / 64 + t with |t| <= 1/128: 2^-(n/64) from a table, 2^-t - 1 by a short series in f32.  The series' rounding is
// 2^-24 of a value below 0.0055, so that a weight is off by 2^-31 of itself: where a prefix's sum or a border falls
// between two of a hundred thousand tokens is then what exact weights would say but for one case in some 10^5 (f32
// weights would be off in one of hundreds).  The likeliest token's weight is exactly 2^45, and 2^18 of it fit 64 bits.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace tq2 {

constexpr int kMaxVocab = 1 << 18;
constexpr int kWeightBits = 45;
constexpr int kBinsPerUnit = 32;  // of log2 of the weight

// 2^-(j/64) in units of 2^-62.
__device__ __forceinline__ uint64_t weight_table_entry(int j) {
    // 2^-(1/64), 2^-(1/32), .. 2^-(1/2)
    constexpr double root[6] = {0.98922801319397548, 0.97857206208770009, 0.95760328069857365,
                                0.91700404320467122, 0.84089641525371454, 0.70710678118654752};
    double v = 1.0;
#pragma unroll
    for (int b = 0; b < 6; ++b)
        if (j >> b & 1) v *= root[b];
    return uint64_t(v * 4611686018427387904.0);
}

// Fills table[64] (shared memory); the caller synchronises the block.
__device__ __forceinline__ void fill_weight_table(uint64_t *table) {
    if (threadIdx.x < 64) table[threadIdx.x] = weight_table_entry(threadIdx.x);
}

struct RowWeights {
    float top;       // the largest logit
    float s_hi, s_lo;  // log2(e) / temperature
    int mode;        // 0: as above, 1: the largest only (no temperature, or an infinite logit)

    __device__ __forceinline__ RowWeights(float largest, float temperature) : top(largest) {
        const double s = 1.4426950408889634 / double(temperature);
        s_hi = float(s);
        s_lo = float(s - double(s_hi));
        mode = !(temperature > 0.f) || s > 1e30 || top == INFINITY;
    }

    // y rounded to f32: larger logits never have a larger one.  (Infinite or NaN: no weight.)
    __device__ __forceinline__ float coarse(float l) const {
        if (mode) return l == top ? 0.f : INFINITY;
        return (top - l) * s_hi;
    }
    // Whether l's coarse y is below `limit` (at most kWeightBits + 1).
    __device__ __forceinline__ bool above(float l, float limit) const { return coarse(l) < limit; }
    // The bin that its coarse y lies in; -1: no weight.
    __device__ __forceinline__ int bin(float l) const {
        const float y = coarse(l);
        return y < float(kWeightBits + 1) ? int(y * float(kBinsPerUnit)) : -1;
    }

    __device__ __forceinline__ uint64_t weight(float l, const uint64_t *table) const {
        if (!(l > -INFINITY)) return 0;  // NaN too
        if (mode) return l == top ? uint64_t(1) << kWeightBits : 0;
        // max - l as hi + lo, exactly
        const float hi = top - l, v = hi - top;
        const float lo = (top - (hi - v)) - (l + v);
        const float p = hi * s_hi;
        if (!(p < float(kWeightBits + 1))) return 0;
        const float e = fmaf(hi, s_hi, -p) + fmaf(hi, s_lo, lo * s_hi);
        const float n = rintf(p * 64.f);
        const float t = fmaf(n, -1.f / 64.f, p) + e;
        // 2^-t - 1 = z + z^2/2 + z^3/6 + z^4/24, z = -t ln 2
        const float z = t * -0.69314718f;
        const float m = z * fmaf(z, fmaf(z, fmaf(z, 1.f / 24.f, 1.f / 6.f), 0.5f), 1.f);
        const int k = int(n);
        const uint64_t base = table[k & 63];
        const int64_t more = __float2ll_rn(__ull2float_rn(base) * m);
        const int shift = 62 - kWeightBits + (k >> 6);
        return (uint64_t(int64_t(base) + more) + (uint64_t(1) << (shift - 1))) >> shift;
    }
};

// A prefix holds a share p of `total` when its mass is this or more (one token at least).
__device__ __forceinline__ uint64_t mass_needed(float p, uint64_t total) {
    const double need = ceil(double(p) * double(total));
    return need >= 1.0 ? min(uint64_t(need), total) : 1;
}
// The smallest weight that min_p keeps; the likeliest token always stays.
__device__ __forceinline__ uint64_t least_weight(float p) {
    const double least = ceil(double(p) * double(uint64_t(1) << kWeightBits));
    return least >= 1.0 ? min(uint64_t(least), uint64_t(1) << kWeightBits) : 0;
}
// The mass that the drawn token's prefix passes: u of `total`, below it.
__device__ __forceinline__ uint64_t drawn_mass(float u, uint64_t total) {
    const double d = floor(double(u) * double(total));
    return d >= 1.0 ? min(uint64_t(d), total - 1) : 0;
}

}  // namespace tq2
