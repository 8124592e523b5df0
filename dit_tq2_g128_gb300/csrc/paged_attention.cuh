// What the two paged attention kernels share: the cache's tensor maps and copies,
// 16-bit packing, values that are not finite, and the join of partial results.
#pragma once

#include <algorithm>

#include <cuda_bf16.h>

#include "tq2_internal.cuh"

namespace tq2 {

template <typename T>
constexpr bool is_half = false;
template <>
constexpr bool is_half<__half> = true;

// log2 of what the softmax's weights are multiplied by before they are rounded to T for the second product (l sums the
// same multiples, so it cancels).  binary16 holds 2^-24 to 65504: weights as they are, at most 2^8 where the maximum
// lags, lose bits below 2^-14 and are gone below 2^-25 of the largest; 2^7 more uses the range to its end.  (A weight of
// 2^-19 was off by 1.8 %, in an f32 output too.)  bf16 has f32's range.
template <typename T>
constexpr float weight_lift = is_half<T> ? 7.f : 0.f;

// Keys from the first token's window to the last token, at most, with what a block of 128
// may hold before them.
inline int64_t key_span(int64_t max_q, int64_t max_kv, int64_t window) {
    return window && window < max_kv ? std::min(max_kv, window + max_q + 126) : max_kv;
}

// 2^x by the hardware approximation (relative error about 2^-22; 2^-inf = 0)
__device__ __forceinline__ float fast_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint64_t drain_ns(uint64_t wait_ns) { return wait_ns > 1000000000ull ? wait_ns : 1000000000ull; }

__device__ __forceinline__ void mbar_expect_tx(uint64_t *bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}

// A value that every lane of the warp holds, told to the compiler to be so.
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

__device__ __forceinline__ bool elect_one() {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
    return ok != 0;
}

// Bounded wait that also ends when another role of the CTA has given up; false (with
// the flag set) then.  The flag and the timer are read at every 64th poll only (read
// at each one, 512 tokens over 32768 keys took 208 us, not 198): a poll that fails
// sleeps for 3.7 us, so a limit is kept to a quarter of a millisecond.
__device__ __forceinline__ bool wait_phase(uint64_t *bar, uint32_t parity, volatile int *abort_flag, uint64_t wait_ns,
                                           unsigned int *status) {
    const uint32_t addr = smem_u32(bar);
    uint64_t t0 = 0;
    for (uint32_t it = 0;; ++it) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(addr), "r"(parity)
            : "memory");
        if (ok) return true;
        if ((it & 63u) == 63u) {
            if (*abort_flag) return false;
            const uint64_t t = globaltimer_ns();
            if (t0 == 0) t0 = t;
            if (t - t0 >= wait_ns) {
                atomicOr(status, static_cast<unsigned int>(TQ2_ERR_TIMEOUT));
                *abort_flag = 1;
                return false;
            }
        }
    }
}

// rows of one page: feature x (a multiple of 64), head, slot, page
__device__ __forceinline__ void tma_cache(uint32_t dst, const CUtensorMap *map, int x, int head, int slot, int page,
                                          uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(head), "r"(slot), "r"(page), "r"(smem_u32(bar))
        : "memory");
}

// One lane issues the copies, from values that the compiler knows to be uniform: spread
// over the lanes, a copy's issue took 50 cycles more.
// The boxes (rows inside one page) of successive tiles of `keys` keys from key0 on, as
// one warp copies them.  The table is read 32 boxes at a time, one window ahead of
// its use: read tile by tile, its latency paced the copies (0.9 us a 64-key tile).
// Tiles of more than 16 boxes (boxes of one or two rows) are looked up as they come.
struct BoxPages {
    const PagedArgs &a;
    const int b, key0, keys, rows, first, last, per, lane;
    int window = -1, now = 0, next = 0;  // table entries of this lane's box in windows `window` and `window` + 1

    __device__ __forceinline__ BoxPages(const PagedArgs &args, int seq, int key_from, int tile_keys, int box_rows, int first_key,
                                        int last_key)
        : a(args), b(seq), key0(uniform(key_from)), keys(tile_keys), rows(box_rows), first(uniform(first_key)),
          last(uniform(last_key)), per(tile_keys / box_rows), lane(int(threadIdx.x & 31)) {}
    __device__ __forceinline__ int entry_of(int box) const {
        const int key = key0 + box * rows;
        return key < last && key + rows > first ? a.batch.page_table[int64_t(b) * a.batch.table_stride + key / a.batch.page_size] : 0;
    }
    // Makes the entries of a tile ready (whole warp; tiles in any order within a window, windows forward).
    __device__ __forceinline__ void seek(int tile) {
        if (per > 16) return;
        const int w = tile * per >> 5;
        if (w == window) return;
        now = window >= 0 && w == window + 1 ? next : entry_of(32 * w + lane);
        next = entry_of(32 * w + 32 + lane);
        window = w;
    }
    __device__ __forceinline__ BoxRange range(int tile) const { return boxes_of(key0 + tile * keys, keys, rows, first, last); }
    // copy(row in the tile, slot in the page, page) for each box of the range, by one lane
    template <typename F>
    __device__ __forceinline__ void each(int tile, BoxRange r, bool &bad, F copy) const {
        const bool one = elect_one();
        int slot = (key0 + (tile * per + r.lo) * rows) % a.batch.page_size;
        for (int i = r.lo; i < r.hi; ++i) {
            const int box = tile * per + i;
            int page = per > 16 ? uniform(entry_of(box)) : __shfl_sync(0xffffffffu, now, box & 31);
            if (page < 0 || int64_t(page) >= a.batch.pages) {  // (recorded; past the last page the copy fills in zeros)
                bad = true;
                page = int(a.batch.pages);
            }
            if (one) copy(i * rows, slot, page);
            slot += rows;
            if (slot >= a.batch.page_size) slot = 0;  // (a box ends with its page or before it)
        }
        __syncwarp();
    }
};

template <typename T>
__device__ __forceinline__ uint32_t pack16(float a, float b) {
    uint32_t r;
    if constexpr (is_half<T>)
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    else
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}
template <typename T>
__device__ __forceinline__ void unpack16(uint32_t w, float &a, float &b) {
    if constexpr (is_half<T>) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
        a = f.x;
        b = f.y;
    } else {
        a = __uint_as_float(w << 16);
        b = __uint_as_float(w & 0xffff0000u);
    }
}

// Whether one of eight 16-bit values is infinite or NaN.
template <typename T>
__device__ __forceinline__ bool any_nonfinite(const uint4 &w) {
    constexpr uint32_t e = is_half<T> ? 0x7c00u : 0x7f80u;
    bool found = false;
    for (uint32_t x : {w.x, w.y, w.z, w.w}) found |= (x & e) == e || ((x >> 16) & e) == e;
    return found;
}

// Sets the values of w that are not finite to zero and hands each to add(element, value).
template <typename T, typename F>
__device__ __forceinline__ void take_nonfinite(uint4 &w, F add) {
    constexpr uint32_t e = is_half<T> ? 0x7c00u : 0x7f80u;
    uint32_t x[4] = {w.x, w.y, w.z, w.w};
    for (int i = 0; i < 4; ++i) {
        float a, b;
        unpack16<T>(x[i], a, b);
        if ((x[i] & e) == e) {
            add(2 * i, a);
            x[i] &= 0xffff0000u;
        }
        if (((x[i] >> 16) & e) == e) {
            add(2 * i + 1, b);
            x[i] &= 0x0000ffffu;
        }
    }
    w = make_uint4(x[0], x[1], x[2], x[3]);
}

__device__ __forceinline__ void store4(float *p, float a, float b, float c, float d) {
    *reinterpret_cast<float4 *>(p) = make_float4(a, b, c, d);
}
template <typename T>
__device__ __forceinline__ void store4(T *p, float a, float b, float c, float d) {
    *reinterpret_cast<uint2 *>(p) = make_uint2(pack16<T>(a, b), pack16<T>(c, d));
}

// Tensor maps of the cache's planes: [pages][slots][heads][dim] in the cache's own
// strides, boxes of 64 features of `box_rows` slots with the 128-byte swizzle
// (features past dim are filled with zeros).
template <typename T>
cudaError_t cache_maps(const PagedArgs &a, int box_rows, CUtensorMap *km, CUtensorMap *vm) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return cudaErrorNotSupported;
    const cuuint64_t dims[4] = {cuuint64_t(a.dim), cuuint64_t(a.kv_heads), cuuint64_t(a.batch.page_size),
                                cuuint64_t(a.batch.pages)};
    // (a stride along an axis of one element is never used)
    auto bytes = [&](int64_t s) { return cuuint64_t(s ? s : a.dim) * 2; };
    const cuuint64_t strides[3] = {bytes(a.head_stride), bytes(a.slot_stride), bytes(a.page_stride)};
    const cuuint32_t box[4] = {64, 1, cuuint32_t(box_rows), 1}, step[4] = {1, 1, 1, 1};
    const CUtensorMapDataType type = is_half<T> ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    for (int i = 0; i < 2; ++i)
        if (enc(i ? vm : km, type, 4, const_cast<void *>(i ? a.v : a.k), dims, strides, box, step,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return cudaErrorInvalidValue;
    return cudaSuccess;
}

// Launch that may begin before the work ahead of it in the stream has ended (the
// kernel waits for that work itself before it touches memory).
template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, int threads, int smem, cudaStream_t stream, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(unsigned(threads));
    cfg.dynamicSmemBytes = size_t(smem);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

constexpr int kJoinWarps = 4;

// Joins `count` partial results of (new token t, head h), the i-th at index place(i):
// out = sum_i 2^(m_i - m) O_i / sum_i 2^(m_i - m) l_i.  A warp takes every
// kJoinWarps-th of them with a running maximum, four in flight, and the warps meet in
// their order: the same bits on every call.  Reads what the launch before wrote (mostly
// from L2).  The whole block.
template <typename TO, typename F>
__device__ __forceinline__ void join_partials(const PagedArgs &a, int64_t t, int h, int count, const float *__restrict__ part_o,
                                              const float2 *__restrict__ part_ml, F place, TO *out) {
    __shared__ float sh_o[kJoinWarps][128], sh_m[kJoinWarps], sh_l[kJoinWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool mine = 4 * lane < a.dim;
    float top = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c0 = warp; c0 < count; c0 += 4 * kJoinWarps) {
        float2 ml[4];
        float4 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = c0 + i * kJoinWarps;
            ml[i] = make_float2(-INFINITY, 0.f);
            x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (c < count) {
                const int64_t at = place(c);
                ml[i] = part_ml[at];
                if (mine) x[i] = *reinterpret_cast<const float4 *>(part_o + at * a.dim + 4 * lane);
            }
        }
        const float next = fmaxf(fmaxf(fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x)), top);
        const float keep = top == next ? 1.f : fast_ex2(top - next);
        l *= keep;
        o.x *= keep;
        o.y *= keep;
        o.z *= keep;
        o.w *= keep;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float f = ml[i].x == next ? 1.f : fast_ex2(ml[i].x - next);
            l = fmaf(f, ml[i].y, l);
            o.x = fmaf(f, x[i].x, o.x);
            o.y = fmaf(f, x[i].y, o.y);
            o.z = fmaf(f, x[i].z, o.z);
            o.w = fmaf(f, x[i].w, o.w);
        }
        top = next;
    }
    if (mine) *reinterpret_cast<float4 *>(&sh_o[warp][4 * lane]) = o;
    if (lane == 0) {
        sh_m[warp] = top;
        sh_l[warp] = l;
    }
    __syncthreads();
    if (warp == 0 && mine) {
        float all = sh_m[0];
#pragma unroll
        for (int w = 1; w < kJoinWarps; ++w) all = fmaxf(all, sh_m[w]);
        l = 0.f;
        o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w) {
            const float f = sh_m[w] == all ? 1.f : fast_ex2(sh_m[w] - all);
            const float4 x = *reinterpret_cast<const float4 *>(&sh_o[w][4 * lane]);
            o.x = fmaf(f, x.x, o.x);
            o.y = fmaf(f, x.y, o.y);
            o.z = fmaf(f, x.z, o.z);
            o.w = fmaf(f, x.w, o.w);
            l = fmaf(f, sh_l[w], l);
        }
        const float inv = l == 0.f ? 0.f : 1.f / l;
        store4(out + t * a.out_token + int64_t(h) * a.out_head + 4 * lane, o.x * inv, o.y * inv, o.z * inv, o.w * inv);
    }
}

}  // namespace tq2
