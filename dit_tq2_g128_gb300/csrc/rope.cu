// Rotary positions with several axes, and the same on the way into a paged
// key/value cache.
//
// Mathematics: pair (a, b) of a head is the complex number a + ib, multiplied by
// exp(i position[axis] inv_freq).  The angle is kept as a fraction of a turn in
// 64-bit integers: phase = position * turns mod 2^64 is exact whatever the
// position, and only the nearest quarter turn's remainder (32 bits of it) is
// rounded to f32: the angle is off by at most 2^-23.6 of a radian (an eighth of a turn
// with 24 bits, times a rounded 2 pi) and a sine or cosine by 1e-7 (2^-23.2; every remainder
// of a sample of four million, in a model of this arithmetic).  (Its own short series:
// with the library's sine the 16-bit forms took 15 instructions an element.)
//
// Bound by memory (each element read once and written once): in f32 by its rate, at 16
// bits by its latency too, as twice the arithmetic lies between one set of loads and the
// next.  A thread owns one unit (VP pairs) of one token: it forms the unit's sines once
// and turns it in up to `hpg` heads, the loads of two heads (four where a pack is less
// than 16 bytes) in flight at a time.
// Any strides: the vector width falls back to one element where the pointers,
// strides or pair count do not allow 16 (8) bytes.
//
// Measured: q, k and v of 4608 tokens, 24 heads of 128 in f32, from rows to heads: 58.3 us,
// 86 % of the copy rate.  Prompts of 16,580 tokens into a paged cache, 32 query and 8
// key heads of 128 in bf16: 101 us, 72 % (32 % of the issue slots, 42 % of the warps, waiting for loads).
// One token: 3.2 us on the GPU, its launch.
#include <cuda_bf16.h>

#include "tq2_internal.cuh"

namespace tq2 {
namespace {

constexpr int kRopeThreads = 256;

template <typename T, int VP>
struct alignas(sizeof(T) * VP) Pack {
    T e[VP];
};

// The pack's elements in f32, and back with one rounding each, two at a time where
// there are two (a conversion instruction makes a pair).
template <int VP>
__device__ __forceinline__ void unpack(const Pack<float, VP> &v, float (&x)[VP]) {
#pragma unroll
    for (int i = 0; i < VP; ++i) x[i] = v.e[i];
}
template <int VP>
__device__ __forceinline__ void unpack(const Pack<__half, VP> &v, float (&x)[VP]) {
    if constexpr (VP == 1) {
        x[0] = __half2float(v.e[0]);
    } else {
#pragma unroll
        for (int i = 0; i < VP; i += 2) {
            const float2 f = __half22float2(__halves2half2(v.e[i], v.e[i + 1]));
            x[i] = f.x;
            x[i + 1] = f.y;
        }
    }
}
template <int VP>
__device__ __forceinline__ void unpack(const Pack<__nv_bfloat16, VP> &v, float (&x)[VP]) {
    if constexpr (VP == 1) {
        x[0] = __bfloat162float(v.e[0]);
    } else {
        const uint32_t *w = reinterpret_cast<const uint32_t *>(&v);
#pragma unroll
        for (int i = 0; i < VP; i += 2) {
            x[i] = __uint_as_float(w[i / 2] << 16);
            x[i + 1] = __uint_as_float(w[i / 2] & 0xffff0000u);
        }
    }
}
template <int VP>
__device__ __forceinline__ void store_pack(float *p, const float (&x)[VP]) {
    Pack<float, VP> v;
#pragma unroll
    for (int i = 0; i < VP; ++i) v.e[i] = x[i];
    *reinterpret_cast<Pack<float, VP> *>(p) = v;
}
template <int VP>
__device__ __forceinline__ void store_pack(__half *p, const float (&x)[VP]) {
    if constexpr (VP == 1) {
        *p = __float2half_rn(x[0]);
    } else {
        Pack<__half2, VP / 2> v;
#pragma unroll
        for (int i = 0; i < VP; i += 2) v.e[i / 2] = __floats2half2_rn(x[i], x[i + 1]);
        *reinterpret_cast<Pack<__half2, VP / 2> *>(p) = v;
    }
}
template <int VP>
__device__ __forceinline__ void store_pack(__nv_bfloat16 *p, const float (&x)[VP]) {
    if constexpr (VP == 1) {
        *p = __float2bfloat16_rn(x[0]);
    } else {
        Pack<__nv_bfloat162, VP / 2> v;
#pragma unroll
        for (int i = 0; i < VP; i += 2) v.e[i / 2] = __floats2bfloat162_rn(x[i], x[i + 1]);
        *reinterpret_cast<Pack<__nv_bfloat162, VP / 2> *>(p) = v;
    }
}

// Sine and cosine of 2 pi phase / 2^64.  After the nearest quarter turn is taken off
// as an integer the angle x is within pi/4, where the series to x^9 and x^10 are off
// by at most x^11/11! = 2e-9 and x^12/12! = 2e-10: f32 rounding decides.
__device__ __forceinline__ void turn_sincos(uint64_t phase, float &sn, float &cs) {
    const uint64_t quarter = (phase + (uint64_t(1) << 61)) >> 62;
    const int64_t rest = int64_t(phase - (quarter << 62));  // [-2^61, 2^61): an eighth of a turn each way
    const float x = float(int32_t(rest >> 30)) * (6.28318530717958648f * 0x1p-34f), z = x * x;
    const float s = fmaf(x * z, fmaf(z, fmaf(z, fmaf(z, 1.f / 362880.f, -1.f / 5040.f), 1.f / 120.f), -1.f / 6.f), x);
    const float c = fmaf(z, fmaf(z, fmaf(z, fmaf(z, fmaf(z, -1.f / 3628800.f, 1.f / 40320.f), -1.f / 720.f), 1.f / 24.f), -0.5f), 1.f);
    const uint32_t q = uint32_t(quarter);
    const bool swap = q & 1;
    // sine's sign is the second bit of q, cosine's that of q + 1
    sn = __uint_as_float(__float_as_uint(swap ? c : s) ^ ((q & 2) << 30));
    cs = __uint_as_float(__float_as_uint(swap ? s : c) ^ (((q + 1) & 2) << 30));
}

// (a, b) times cos + i sin
__device__ __forceinline__ void turn(float &a, float &b, float cs, float sn) {
    const float x = a;
    a = fmaf(x, cs, -b * sn);
    b = fmaf(x, sn, b * cs);
}

// grid: x = tokens * units / threads, y = head groups of all segments
template <typename TI, typename TO, int VP>
__global__ void __launch_bounds__(kRopeThreads, 4)
rope_kernel(const RopeArgs a, int units, int hpg, unsigned int *status) {
    const int64_t idx = int64_t(blockIdx.x) * kRopeThreads + threadIdx.x;
    int64_t t;
    int u;
    if (idx <= 0xffffffffll) {
        t = uint32_t(idx) / uint32_t(units);
        u = int(uint32_t(idx) - uint32_t(t) * uint32_t(units));
    } else {
        t = idx / units;
        u = int(idx - t * units);
    }
    if (t >= a.tokens) return;
    int s = 0, group = blockIdx.y;
    for (; s < a.nseg - 1; ++s) {
        const int n = (a.seg[s].heads + hpg - 1) / hpg;
        if (group < n) break;
        group -= n;
    }
    const RopeSegment &g = a.seg[s];

    // where this token goes
    int64_t key = 0;
    int64_t out_base = t * g.out_token;
    if (a.append) {
        const int b = seq_of(a.batch, t);
        if (b < 0) return;
        bool bad = false;
        const SeqSpan sp = seq_span(a.batch, b, bad);
        report_bad(bad, status);
        if (t < sp.q0 || t >= int64_t(sp.q0) + sp.n || (bad && g.paged)) return;  // (clamped lengths would name the slots of older keys)
        key = int64_t(sp.kv) - sp.n + (t - sp.q0);
        if (g.paged) {
            if (key < 0) return;
            const int in_table = int(key) / a.batch.page_size;
            const int64_t page = page_of(a.batch, b, in_table, bad);
            report_bad(bad, status);
            if (page < 0) return;
            out_base = page * a.page_stride + int64_t(int(key) - in_table * a.batch.page_size) * g.out_token;
        }
    }

    // the unit's two packs of VP elements in each head
    const int ru = a.pairs / VP;  // units that are turned
    const bool turned = g.turned && u < ru;
    int e0, e1;
    if (g.turned && u < ru) {
        e0 = a.interleaved ? u * 2 * VP : u * VP;
        e1 = a.interleaved ? e0 + VP : a.pairs + e0;
    } else {
        e0 = g.turned ? 2 * a.pairs + (u - ru) * 2 * VP : u * 2 * VP;
        e1 = e0 + VP;
    }
    const bool has0 = VP > 1 || e0 < a.dim, has1 = VP > 1 || e1 < a.dim;  // (a scalar copy unit may end inside)
    const int h0 = group * hpg, count = min(hpg, g.heads - h0);
    const TI *in = static_cast<const TI *>(g.in) + t * g.in_token + int64_t(h0) * g.in_head + e0;
    TO *out = static_cast<TO *>(g.out) + out_base + int64_t(h0) * g.out_head + e0;
    const int64_t in_step = g.in_head, out_step = g.out_head;
    const int gap = e1 - e0;
    constexpr int HF = sizeof(TI) * VP >= 16 ? 2 : 4;  // heads in flight
    Pack<TI, VP> x[HF], y[HF];
    auto load = [&](int left) {  // the next heads, `in` past them
#pragma unroll
        for (int j = 0; j < HF; ++j) {
            if (j < left) {
                if (has0) x[j] = *reinterpret_cast<const Pack<TI, VP> *>(in);
                if (has1) y[j] = *reinterpret_cast<const Pack<TI, VP> *>(in + gap);
            }
            in += in_step;
        }
    };
    load(count);
    float sn[VP], cs[VP];
    if (turned) {
        int64_t pos = a.positions ? 0 : key;
        int axis = -1;
#pragma unroll
        for (int i = 0; i < VP; ++i) {
            const int p = u * VP + i;
            if (a.positions) {
                const int ax = a.axis ? min(int(a.axis[p]), a.axes - 1) : 0;
                if (ax != axis) pos = a.positions[t * a.axes + ax];
                axis = ax;
            }
            turn_sincos(uint64_t(pos) * a.turns[p], sn[i], cs[i]);
            if (a.inverse) sn[i] = -sn[i];
        }
    }
#pragma unroll 1
    for (int left = count; left > 0; left -= HF) {
        if (left < count) load(left);
#pragma unroll
        for (int j = 0; j < HF; ++j) {
            if (j < left) {
                float r0[VP], r1[VP];
                unpack(x[j], r0);
                unpack(y[j], r1);
                if (turned) {
                    if (VP == 1 || !a.interleaved) {
#pragma unroll
                        for (int i = 0; i < VP; ++i) turn(r0[i], r1[i], cs[i], sn[i]);
                    } else {  // pairs lie inside each pack: angles 0 .. VP/2 - 1, then the rest
#pragma unroll
                        for (int i = 0; i < VP / 2; ++i) {
                            turn(r0[2 * i], r0[2 * i + 1], cs[i], sn[i]);
                            turn(r1[2 * i], r1[2 * i + 1], cs[VP / 2 + i], sn[VP / 2 + i]);
                        }
                    }
                }
                if (has0) store_pack<VP>(out, r0);
                if (has1) store_pack<VP>(out + gap, r1);
            }
            out += out_step;
        }
    }
}

// pointers, strides and pair count allow packs of vp elements
bool packs(const RopeArgs &a, int vp, int in_bytes, int out_bytes) {
    if (a.pairs % vp || a.dim % (2 * vp)) return false;
    for (int s = 0; s < a.nseg; ++s) {
        const RopeSegment &g = a.seg[s];
        if (reinterpret_cast<uintptr_t>(g.in) % (vp * in_bytes) || reinterpret_cast<uintptr_t>(g.out) % (vp * out_bytes))
            return false;
        if (g.in_token % vp || g.in_head % vp || g.out_token % vp || g.out_head % vp) return false;
        if (g.paged && a.page_stride % vp) return false;
    }
    return true;
}

template <typename TI, typename TO, int VP>
cudaError_t launch_rope_vp(const RopeArgs &a, const LaunchCtx &ctx) {
    const int units = VP == 1 ? a.pairs + (a.dim - 2 * a.pairs + 1) / 2 : a.dim / (2 * VP);
    // heads per thread: as many (up to 16, for the sines' sake) as leave every SM its threads
    int all = 0;
    for (int s = 0; s < a.nseg; ++s) all += a.seg[s].heads;
    int hpg = 16;
    while (hpg > 1 && a.tokens * units * ((all + hpg - 1) / hpg) < int64_t(ctx.num_sms) * 2048) hpg >>= 1;
    int groups = 0;
    for (int s = 0; s < a.nseg; ++s) groups += (a.seg[s].heads + hpg - 1) / hpg;
    if (groups == 0) return cudaSuccess;
    const int64_t blocks = (a.tokens * units + kRopeThreads - 1) / kRopeThreads;
    if (blocks > INT32_MAX || groups > 65535) return cudaErrorInvalidValue;
    rope_kernel<TI, TO, VP><<<dim3(unsigned(blocks), unsigned(groups)), kRopeThreads, 0, ctx.stream>>>(a, units, hpg,
                                                                                                       ctx.status);
    return cudaPeekAtLastError();
}

template <typename TI, typename TO>
cudaError_t launch_rope_io(const RopeArgs &a, const LaunchCtx &ctx) {
    if constexpr (sizeof(TI) == 2 && sizeof(TO) == 2)
        if (packs(a, 8, 2, 2)) return launch_rope_vp<TI, TO, 8>(a, ctx);
    if (packs(a, 4, sizeof(TI), sizeof(TO))) return launch_rope_vp<TI, TO, 4>(a, ctx);
    return launch_rope_vp<TI, TO, 1>(a, ctx);
}

template <typename TI>
cudaError_t launch_rope_in(const RopeArgs &a, int out_dtype, const LaunchCtx &ctx) {
    switch (out_dtype) {
        case TQ2_F32: return launch_rope_io<TI, float>(a, ctx);
        case TQ2_F16: return launch_rope_io<TI, __half>(a, ctx);
        default: return launch_rope_io<TI, __nv_bfloat16>(a, ctx);
    }
}

}  // namespace

cudaError_t launch_rope(const RopeArgs &a, int in_dtype, int out_dtype, const LaunchCtx &ctx) {
    switch (in_dtype) {
        case TQ2_F32: return launch_rope_in<float>(a, out_dtype, ctx);
        case TQ2_F16: return launch_rope_in<__half>(a, out_dtype, ctx);
        default: return launch_rope_in<__nv_bfloat16>(a, out_dtype, ctx);
    }
}

}  // namespace tq2
