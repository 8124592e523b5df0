// The weight of a token in sampling, as an integer in units of 2^-45 of the likeliest token's.
//
// w = 2^-y, y = (max - l) log2(e) / temperature.  y is kept as a sum of two f32 (its error is 2^-46 of it), split into
// n / 64 + t with |t| <= 1/128: 2^-(n/64) from a table, 2^-t - 1 by a short series in f32.  The roundings of t, of the series
// and of its product with the table's entry are half a step each of values below 0.0055: at most 5.5 * 2^-32 together, so that a
// weight is within 2^-29.5 of itself (2^-31 as a rule) and half a unit.  Where a prefix's sum or a border falls
// between two of a hundred thousand tokens is then what exact weights would say but for one case in some 10^5 (f32
// weights would be off in one of hundreds).  The likeliest token's weight is exactly 2^45, and 2^18 of it fit 64 bits.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace tq2 {

constexpr int kMaxVocab = 1 << 18;
constexpr int kWeightBits = 45;

// 2^-(j/64) in units of 2^-62, to 53 bits.
struct WeightTable {
    uint64_t e[64];
};
constexpr WeightTable make_weight_table() {
    // 2^-(1/64), 2^-(1/32), .. 2^-(1/2)
    constexpr double root[6] = {0.98922801319397548, 0.97857206208770009, 0.95760328069857365,
                                0.91700404320467122, 0.84089641525371454, 0.70710678118654752};
    WeightTable t = {};
    for (int j = 0; j < 64; ++j) {
        double v = 1.0;
        for (int b = 0; b < 6; ++b)
            if (j >> b & 1) v *= root[b];
        t.e[j] = uint64_t(v * 4611686018427387904.0);
    }
    return t;
}
__constant__ WeightTable weight_table = make_weight_table();

// A row's weights.  In f32 and integers throughout: 64-bit floating point, and conversions to and from it, run at a
// thirtieth of their rate.  No branches: a weight is a chain of some 60 instructions, and several have to be under way (with
// branches between them a pass over 49 elements a thread took 15,000 cycles).
struct RowWeights {
    float top;         // the largest logit
    float s_hi, s_lo;  // log2(e) / temperature
    bool only;         // the largest only (no temperature, or an infinite logit): s_hi is infinite

    __device__ __forceinline__ RowWeights(float largest, float temperature) : top(largest) {
        constexpr float e_hi = 1.44269502f, e_lo = 1.92596303e-8f;  // log2(e)
        s_hi = e_hi / temperature;
        s_lo = (fmaf(-s_hi, temperature, e_hi) + e_lo) / temperature;
        only = !(temperature > 0.f) || !(s_hi < 1e30f) || top == INFINITY;
        if (!(temperature < INFINITY)) s_hi = s_lo = 0.f;
        if (only) {
            s_hi = INFINITY;
            s_lo = 0.f;
        }
    }

    // y rounded to f32: larger logits never have a larger one.  (Infinite or NaN: no weight.)
    __device__ __forceinline__ float coarse(float l) const {
        return l == top ? 0.f : (top - l) * s_hi;
    }
    // A logit below which no token has a coarse y below `limit`.
    __device__ __forceinline__ float floor_of(float limit) const {
        return only ? top : fmaxf(top - limit * (1.f + 0x1p-18f) / s_hi, -3.402823466e38f);
    }

    __device__ __forceinline__ uint64_t weight(float l, const uint64_t *table) const {
        // max - l as hi + lo, exactly
        const float hi = top - l, v = hi - top;
        const float lo = (top - (hi - v)) - (l + v);
        const float y = hi * s_hi, p = fminf(y, float(kWeightBits + 1));  // (of -inf and NaN: infinite or NaN, and no weight)
        const float e = fmaf(hi, s_hi, -p) + fmaf(hi, s_lo, lo * s_hi);
        // n = 64 p to the nearest integer, in the low bits of its sum with 1.5 * 2^23
        const float big = fmaf(p, 64.f, 12582912.f);
        const int k = __float_as_int(big) - __float_as_int(12582912.f);
        const float t = fmaf(big - 12582912.f, -1.f / 64.f, p) + e;
        // 2^-t - 1 = z + z^2/2 + z^3/6 + z^4/24, z = -t ln 2
        const float z = t * -0.69314718f;
        const float m = z * fmaf(z, fmaf(z, fmaf(z, 1.f / 24.f, 1.f / 6.f), 0.5f), 1.f);
        const uint64_t base = table[k & 63];
        // base (2^-62) times m, below 2^-7: to 2^-38 in 32 bits
        const float high = __uint2float_rn(uint32_t(base >> 32)) * m;
        const int64_t more = int64_t(__float2int_rn(high * 256.f)) * (1 << 24);
        const int shift = 62 - kWeightBits + (k >> 6);
        const uint64_t w = (base + uint64_t(more) + (uint64_t(1) << (shift - 1))) >> shift;
        return l == top ? uint64_t(1) << kWeightBits : y < float(kWeightBits + 1) ? w : 0;
    }
};

// floor(f * total) for 0 <= f < 1, exactly; rest: whether anything was cut off.
__device__ __forceinline__ uint64_t share(float f, uint64_t total, bool *rest) {
    const uint32_t bits = __float_as_uint(f), e = bits >> 23;
    const uint64_t m = e ? (bits & 0x7fffffu) | 0x800000u : bits & 0x7fffffu;  // f = m 2^-down
    const uint32_t down = e ? 150 - e : 149;
    const uint64_t lo = m * total, hi = __umul64hi(m, total);
    *rest = f > 0.f;
    if (down >= 128) return 0;
    if (down >= 64) {
        *rest = lo || (hi & ((uint64_t(1) << (down - 64)) - 1));
        return hi >> (down - 64);
    }
    *rest = lo & ((uint64_t(1) << down) - 1);
    return hi << (64 - down) | lo >> down;  // (f < 1: down is 24 or more)
}
// A prefix holds a share p < 1 of `total` when its mass is this or more (one token at least).
__device__ __forceinline__ uint64_t mass_needed(float p, uint64_t total) {
    if (!(p > 0.f)) return 1;
    bool rest;
    const uint64_t need = share(p, total, &rest) + rest;
    return need ? need : 1;
}
// The smallest weight that min_p keeps; the likeliest token always stays.
__device__ __forceinline__ uint64_t least_weight(float p) {
    if (!(p > 0.f)) return 0;
    if (p >= 1.f) return uint64_t(1) << kWeightBits;
    bool rest;
    const uint64_t least = share(p, uint64_t(1) << kWeightBits, &rest);
    return least + rest;
}
// The mass that the drawn token's prefix passes: u of `total`, below it.
__device__ __forceinline__ uint64_t drawn_mass(float u, uint64_t total) {
    if (!(u > 0.f)) return 0;
    if (u >= 1.f) return total - 1;
    bool rest;
    return share(u, total, &rest);
}

}  // namespace tq2
