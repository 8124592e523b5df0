// C-ABI entry points: host-side validation, kernel choice by shape, launch.
//
// The contract follows "oxibonsai-image 0.2.2 src/gpu.rs" (`ternary_matmul_gpu`
// and its module doc "Correctness contract"): row-major f32 input[M,K],
// out-major TQ2_0_g128 weight blocks [N, K/128], f32 out[M,N] written in full,
// K a multiple of 128.  Unlike the page, every failure is a returned status
// and there is no CPU fallback.
#include <atomic>
#include <cmath>
#include <initializer_list>
#include <cstdint>
#include <cstring>
#include <mutex>

#include "tq2_internal.cuh"

namespace {

// Device status word: kernels OR TQ2_ERR_TIMEOUT into it when a bounded wait
// gives up, TQ2_ERR_BAD_BATCH (a bit of its own) when a batch's tables are out of range.  Static device memory of this module (one word per device).
__device__ unsigned int g_device_status;

std::atomic<uint64_t> g_wait_ns{2000000000ull};

constexpr int kMaxDevices = 64;
struct DeviceInfo {
    int checked = 0;    // 0 = not yet, 1 = supported, -1 = unsupported
    int num_sms = 0;
    unsigned int *status = nullptr;
};
DeviceInfo g_dev[kMaxDevices];
std::mutex g_dev_mu;

// Looks up (once per device) whether the current device is sm_103 and where
// its status word lives.
int current_device(DeviceInfo *out) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return TQ2_ERR_CUDA;
    if (dev < 0 || dev >= kMaxDevices) return TQ2_ERR_UNSUPPORTED_DEVICE;
    std::lock_guard<std::mutex> lock(g_dev_mu);
    DeviceInfo &d = g_dev[dev];
    if (d.checked == 0) {
        int major = 0, minor = 0, sms = 0;
        if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return TQ2_ERR_CUDA;
        if (major != 10 || minor != 3) {
            d.checked = -1;
        } else {
            void *p = nullptr;
            if (cudaGetSymbolAddress(&p, g_device_status) != cudaSuccess) return TQ2_ERR_CUDA;
            d.status = static_cast<unsigned int *>(p);
            d.num_sms = sms;
            d.checked = 1;
        }
    }
    if (d.checked < 0) return TQ2_ERR_UNSUPPORTED_DEVICE;
    *out = d;
    return TQ2_OK;
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Every operand a kernel reads or writes (through plain accesses, tensor maps,
// bulk copies or the tensor kernels' cluster-multicast copies) must be device
// memory of the current device: host memory, managed memory and another
// GPU's memory (peer or imported mappings) are refused before any launch.
// NULL pointers pass (the callers check them where they are required).
bool on_current_device(const void *p, int dev) {
    if (!p) return true;
    cudaPointerAttributes a;
    if (cudaPointerGetAttributes(&a, p) != cudaSuccess) {
        (void)cudaGetLastError();  // not a pointer the runtime knows: not device memory
        return false;
    }
    return a.type == cudaMemoryTypeDevice && a.device == dev;
}

int check_local(std::initializer_list<const void *> ptrs) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return TQ2_ERR_CUDA;
    for (const void *p : ptrs)
        if (!on_current_device(p, dev)) return TQ2_ERR_INVALID_ARG;
    return TQ2_OK;
}

bool overlaps(const void *a, size_t na, const void *b, size_t nb) {
    uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return na && nb && x < y + nb && y < x + na;
}

// Shape-only checks.  Returns TQ2_OK and sets *noop when there is nothing
// to compute.
int check_shape(int64_t m, int64_t n, int64_t k, bool *noop) {
    *noop = false;
    if (k <= 0 || k % tq2::kBlockW) return TQ2_ERR_BAD_K;
    if (m < 0 || n < 0) return TQ2_ERR_INVALID_ARG;
    const int64_t lim = int64_t(1) << 40;  // element counts beyond this are rejected
    if (k > lim || m > lim || n > lim || (m && k > lim / m) || (n && k > lim / n) ||
        (m && n > lim / m))
        return TQ2_ERR_INVALID_ARG;
    if (m == 0 || n == 0) *noop = true;
    return TQ2_OK;
}

// Shape and pointer checks shared by every matmul entry point.
int check_matmul(const void *w, const float *x, const float *residual, const float *out,
                 int64_t m, int64_t n, int64_t k, bool *noop) {
    int st = check_shape(m, n, k, noop);
    if (st != TQ2_OK || *noop) return st;
    if (!w || !x || !out) return TQ2_ERR_INVALID_ARG;
    if (!aligned16(w) || !aligned16(x) || !aligned16(out) || (residual && !aligned16(residual)))
        return TQ2_ERR_MISALIGNED;
    const size_t wb = size_t(n) * size_t(k / tq2::kBlockW) * tq2::kBlockBytes;
    const size_t xb = size_t(m) * size_t(k) * 4, ob = size_t(m) * size_t(n) * 4;
    if (overlaps(out, ob, x, xb) || overlaps(out, ob, w, wb)) return TQ2_ERR_INVALID_ARG;
    if (residual && residual != out && overlaps(out, ob, residual, ob)) return TQ2_ERR_INVALID_ARG;
    return TQ2_OK;
}

int make_ctx(cudaStream_t stream, tq2::LaunchCtx *ctx) {
    DeviceInfo d;
    int st = current_device(&d);
    if (st != TQ2_OK) return st;
    ctx->stream = stream;
    ctx->status = d.status;
    ctx->wait_ns = g_wait_ns.load(std::memory_order_relaxed);
    ctx->num_sms = d.num_sms;
    return TQ2_OK;
}

// Launch context for the current device, then the residency check of every
// operand the call's kernels touch (see on_current_device).
int prepare(void *stream, tq2::LaunchCtx *ctx, std::initializer_list<const void *> ptrs) {
    int st = make_ctx(static_cast<cudaStream_t>(stream), ctx);
    if (st != TQ2_OK) return st;
    return check_local(ptrs);
}

int finish(cudaError_t e) { return e == cudaSuccess ? TQ2_OK : TQ2_ERR_CUDA; }

// M at and above which the tcgen05 kernel beats the f32 CUDA-core small-M kernel.
// (measured at K = N = 4096: M=2 15.4 vs 17.6 us, M=3 20.8 vs 17.6 us)
constexpr int64_t kTcMinM = 3;
// Largest M that tq2_gemm sends to the one-launch skinny tensor-core kernel.
constexpr int64_t kSkinnyMmaMaxM = 32;

}  // namespace

extern "C" {

size_t tq2_soa_bytes(int64_t n, int64_t k) {
    if (n < 0 || k <= 0 || k % tq2::kBlockW) return 0;
    return size_t(n) * size_t(k / tq2::kBlockW) * tq2::kBlockBytes;
}

const char *tq2_status_string(int status) {
    switch (status) {
        case TQ2_OK: return "TQ2_OK";
        case TQ2_ERR_INVALID_ARG: return "TQ2_ERR_INVALID_ARG: null pointer, negative size, overlap or size overflow";
        case TQ2_ERR_BAD_K: return "TQ2_ERR_BAD_K: k must be a positive multiple of 128";
        case TQ2_ERR_MISALIGNED: return "TQ2_ERR_MISALIGNED: device pointers must be 16-byte aligned";
        case TQ2_ERR_UNSUPPORTED_DEVICE: return "TQ2_ERR_UNSUPPORTED_DEVICE: needs compute capability 10.3 (sm_103a)";
        case TQ2_ERR_CUDA: return "TQ2_ERR_CUDA: CUDA launch or runtime error";
        case TQ2_ERR_TIMEOUT: return "TQ2_ERR_TIMEOUT: a bounded device-side wait expired";
        case TQ2_ERR_TOO_LARGE: return "TQ2_ERR_TOO_LARGE: the shape needs more scratch than tq2_gemm_noalloc has";
        case TQ2_ERR_BAD_BATCH: return "TQ2_ERR_BAD_BATCH: a length, offset or page in a batch's device tables is out of range";
        default: return "unknown tq2 status";
    }
}

int tq2_version(void) { return 0x000100; }

uint64_t tq2_set_wait_timeout_ns(uint64_t ns) { return g_wait_ns.exchange(ns); }

int tq2_device_status(void *stream) {
    DeviceInfo d;
    int st = current_device(&d);
    if (st != TQ2_OK) return st;
    if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return TQ2_ERR_CUDA;
    unsigned int v = 0;
    if (cudaMemcpy(&v, d.status, sizeof(v), cudaMemcpyDeviceToHost) != cudaSuccess) return TQ2_ERR_CUDA;
    // what is reported is cleared; the other kind waits for the next call
    st = (v & TQ2_ERR_TIMEOUT) == TQ2_ERR_TIMEOUT ? TQ2_ERR_TIMEOUT : v & TQ2_ERR_BAD_BATCH ? TQ2_ERR_BAD_BATCH : TQ2_OK;
    const unsigned int left = st == TQ2_ERR_TIMEOUT ? v & TQ2_ERR_BAD_BATCH : 0;
    if (cudaMemcpy(d.status, &left, sizeof(left), cudaMemcpyHostToDevice) != cudaSuccess) return TQ2_ERR_CUDA;
    return st;
}

int tq2_select_kernel(int64_t m, int64_t n, int64_t k) {
    if (m == 1) return TQ2_KERNEL_GEMV;
    if (m <= kSkinnyMmaMaxM && tq2::skinny_mma_fits(m, n, k)) return TQ2_KERNEL_SKINNY_MMA;
    if (m < kTcMinM && m <= tq2::kSkinnyMaxM) return TQ2_KERNEL_SKINNY;
    return TQ2_KERNEL_TC;
}

int tq2_reformat_aos_to_soa(const void *w_aos, void *w_soa, int64_t n, int64_t k, void *stream) {
    if (k <= 0 || k % tq2::kBlockW) return TQ2_ERR_BAD_K;
    if (n < 0 || n > (int64_t(1) << 40) / (k / tq2::kBlockW)) return TQ2_ERR_INVALID_ARG;
    if (n == 0) return TQ2_OK;
    if (!w_aos || !w_soa) return TQ2_ERR_INVALID_ARG;
    if (!aligned16(w_soa)) return TQ2_ERR_MISALIGNED;
    if (overlaps(w_aos, tq2_soa_bytes(n, k), w_soa, tq2_soa_bytes(n, k))) return TQ2_ERR_INVALID_ARG;
    tq2::LaunchCtx ctx;
    int st = prepare(stream, &ctx, {w_aos, w_soa});
    if (st != TQ2_OK) return st;
    return finish(tq2::launch_reformat(w_aos, w_soa, n, k, ctx));
}

int tq2_quantize_f32(const float *w, void *w_aos, int64_t n, int64_t k, void *stream) {
    if (k <= 0 || k % tq2::kBlockW) return TQ2_ERR_BAD_K;
    if (n < 0 || n > (int64_t(1) << 40) / k) return TQ2_ERR_INVALID_ARG;
    if (n == 0) return TQ2_OK;
    if (!w || !w_aos) return TQ2_ERR_INVALID_ARG;
    if (!aligned16(w) || !aligned16(w_aos)) return TQ2_ERR_MISALIGNED;
    if (overlaps(w, size_t(n) * size_t(k) * 4, w_aos, tq2_soa_bytes(n, k))) return TQ2_ERR_INVALID_ARG;
    tq2::LaunchCtx ctx;
    int st = prepare(stream, &ctx, {w, w_aos});
    if (st != TQ2_OK) return st;
    return finish(tq2::launch_quantize(w, w_aos, n, k, ctx));
}

int tq2_gemm_with(int kernel, const void *w_soa, const float *x, const float *residual,
                  float *out, int64_t m, int64_t n, int64_t k, void *stream) {
    bool noop = false;
    int st = check_matmul(w_soa, x, residual, out, m, n, k, &noop);
    if (st != TQ2_OK || noop) return st;
    if (kernel == TQ2_KERNEL_AUTO) kernel = tq2_select_kernel(m, n, k);
    if (kernel == TQ2_KERNEL_GEMV && m != 1) return TQ2_ERR_INVALID_ARG;
    if (kernel == TQ2_KERNEL_SKINNY && m > tq2::kSkinnyMaxM) return TQ2_ERR_INVALID_ARG;
    if (kernel == TQ2_KERNEL_SKINNY_MMA && !tq2::skinny_mma_fits(m, n, k)) return TQ2_ERR_INVALID_ARG;
    if (kernel < TQ2_KERNEL_GEMV || kernel > TQ2_KERNEL_SKINNY_MMA) return TQ2_ERR_INVALID_ARG;
    tq2::LaunchCtx ctx;
    st = prepare(stream, &ctx, {w_soa, x, residual, out});
    if (st != TQ2_OK) return st;
    switch (kernel) {
        case TQ2_KERNEL_GEMV: return finish(tq2::launch_gemv(w_soa, x, residual, out, n, k, ctx));
        case TQ2_KERNEL_SKINNY:
            return finish(tq2::launch_skinny(w_soa, x, residual, out, m, n, k, ctx));
        case TQ2_KERNEL_TC: {
            // x -> f16 tiles in a stream-ordered temporary, then the clustered
            // kernel.  A failed allocation is reported (TQ2_ERR_CUDA, the
            // CUDA error left for the caller), never replaced by another kernel.
            void *ws = nullptr;
            if (cudaMallocAsync(&ws, tq2::tc_ws_bytes(m, n, k), ctx.stream) != cudaSuccess)
                return TQ2_ERR_CUDA;
            const cudaError_t e = tq2::launch_tc_ws(w_soa, x, residual, out, m, n, k, ws, ctx);
            const cudaError_t f = cudaFreeAsync(ws, ctx.stream);
            return finish(e != cudaSuccess ? e : f);
        }
        case TQ2_KERNEL_TC_DIRECT:
            return finish(tq2::launch_tc(w_soa, x, residual, out, m, n, k, ctx));
        case TQ2_KERNEL_SKINNY_MMA:
            return finish(tq2::launch_skinny_mma(w_soa, x, residual, out, m, n, k, ctx));
        default: return finish(tq2::launch_f32ref(w_soa, x, residual, out, m, n, k, ctx));
    }
}

size_t tq2_gemm_workspace_bytes(int64_t m, int64_t n, int64_t k) {
    bool noop = false;
    if (check_shape(m, n, k, &noop) != TQ2_OK || noop) return 0;
    if (tq2_select_kernel(m, n, k) != TQ2_KERNEL_TC) return 0;
    return tq2::tc_ws_bytes(m, n, k);
}

int tq2_gemm_ws(const void *w_soa, const float *x, const float *residual, float *out, int64_t m,
                int64_t n, int64_t k, void *workspace, size_t workspace_bytes, void *stream) {
    bool noop = false;
    int st = check_matmul(w_soa, x, residual, out, m, n, k, &noop);
    if (st != TQ2_OK || noop) return st;
    if (tq2_select_kernel(m, n, k) != TQ2_KERNEL_TC)
        return tq2_gemm_with(TQ2_KERNEL_AUTO, w_soa, x, residual, out, m, n, k, stream);
    const size_t need = tq2::tc_ws_bytes(m, n, k);
    if (!workspace || workspace_bytes < need) return TQ2_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(workspace) & 127u) != 0) return TQ2_ERR_MISALIGNED;
    const size_t wb = size_t(n) * size_t(k / tq2::kBlockW) * tq2::kBlockBytes;
    const size_t xb = size_t(m) * size_t(k) * 4, ob = size_t(m) * size_t(n) * 4;
    if (overlaps(workspace, need, x, xb) || overlaps(workspace, need, w_soa, wb) ||
        overlaps(workspace, need, out, ob) || (residual && overlaps(workspace, need, residual, ob)))
        return TQ2_ERR_INVALID_ARG;
    tq2::LaunchCtx ctx;
    st = prepare(stream, &ctx, {w_soa, x, residual, out, workspace});
    if (st != TQ2_OK) return st;
    return finish(tq2::launch_tc_ws(w_soa, x, residual, out, m, n, k, workspace, ctx));
}

int tq2_gemm_noalloc(const void *w_soa, const float *x, const float *residual, float *out,
                     int64_t m, int64_t n, int64_t k, void *stream) {
    bool noop = false;
    int st = check_matmul(w_soa, x, residual, out, m, n, k, &noop);
    if (st != TQ2_OK || noop) return st;
    if (tq2_select_kernel(m, n, k) != TQ2_KERNEL_TC)  // these kernels use no scratch
        return tq2_gemm_with(TQ2_KERNEL_AUTO, w_soa, x, residual, out, m, n, k, stream);
    // the one place that checks the shape against the fixed scratch; it comes
    // before the device is looked up (a host-only decision, like the other
    // argument checks)
    if (tq2::tc_ws_bytes(m, n, k) > tq2::kNoAllocScratchBytes) return TQ2_ERR_TOO_LARGE;
    tq2::LaunchCtx ctx;
    st = prepare(stream, &ctx, {w_soa, x, residual, out});
    if (st != TQ2_OK) return st;
    return finish(tq2::launch_tc_noalloc(w_soa, x, residual, out, m, n, k, ctx));
}

int tq2_gemm(const void *w_soa, const float *x, const float *residual, float *out, int64_t m,
             int64_t n, int64_t k, void *stream) {
    return tq2_gemm_with(TQ2_KERNEL_AUTO, w_soa, x, residual, out, m, n, k, stream);
}

static int gate_up_swiglu(const void *w_soa, const float *x, float *out, int64_t m, int64_t f,
                          int64_t k, void *stream, bool resident) {
    if (k <= 0 || k % tq2::kBlockW) return TQ2_ERR_BAD_K;
    if (f < 0 || f > (int64_t(1) << 39)) return TQ2_ERR_INVALID_ARG;
    bool noop = false;
    int st = check_shape(m, 2 * f, k, &noop);
    if (st != TQ2_OK || noop) return st;
    if (!w_soa || !x || !out) return TQ2_ERR_INVALID_ARG;
    if (!aligned16(w_soa) || !aligned16(x) || !aligned16(out)) return TQ2_ERR_MISALIGNED;
    const size_t wb = size_t(2 * f) * size_t(k / tq2::kBlockW) * tq2::kBlockBytes;
    const size_t xb = size_t(m) * size_t(k) * 4, ob = size_t(m) * size_t(f) * 4;
    if (overlaps(out, ob, x, xb) || overlaps(out, ob, w_soa, wb)) return TQ2_ERR_INVALID_ARG;
    tq2::LaunchCtx ctx;
    st = prepare(stream, &ctx, {w_soa, x, out});
    if (st != TQ2_OK) return st;
    cudaError_t e = cudaErrorNotSupported;
    if (m == 1) {
        e = tq2::launch_gemv_swiglu(w_soa, x, out, f, k, ctx, resident);
    } else if (f % 16 == 0) {
        void *ws = nullptr;
        if (cudaMallocAsync(&ws, tq2::tc_swiglu_ws_bytes(m, k), ctx.stream) != cudaSuccess) {
            (void)cudaGetLastError();
            return TQ2_ERR_CUDA;
        }
        e = tq2::launch_tc_swiglu(w_soa, x, out, m, f, k, ws, ctx);
        const cudaError_t fr = cudaFreeAsync(ws, ctx.stream);
        if (e == cudaSuccess) e = fr;
    }
    if (e != cudaErrorNotSupported) return finish(e);
    (void)cudaGetLastError();
    // Shapes outside the fused kernels: the plain product into a stream-ordered
    // temporary [m, 2f], then the element-wise activation.
    void *gu = nullptr;
    if (cudaMallocAsync(&gu, size_t(m) * size_t(2 * f) * 4, ctx.stream) != cudaSuccess) {
        (void)cudaGetLastError();
        return TQ2_ERR_CUDA;
    }
    st = tq2_gemm_with(TQ2_KERNEL_AUTO, w_soa, x, nullptr, static_cast<float *>(gu), m, 2 * f, k, stream);
    if (st == TQ2_OK) st = finish(tq2::launch_swiglu_rows(static_cast<const float *>(gu), out, m, f, ctx));
    const cudaError_t fr = cudaFreeAsync(gu, ctx.stream);
    return st != TQ2_OK ? st : finish(fr);
}

int tq2_gate_up_swiglu(const void *w_soa, const float *x, float *out, int64_t m, int64_t f,
                       int64_t k, void *stream) {
    return gate_up_swiglu(w_soa, x, out, m, f, k, stream, false);
}

int tq2_gate_up_swiglu_resident(const void *w_soa, const float *x, float *out, int64_t m, int64_t f,
                                int64_t k, void *stream) {
    return gate_up_swiglu(w_soa, x, out, m, f, k, stream, true);
}

int tq2_act16_from_f32(const float *x, void *x16, int64_t m, int64_t k, void *stream) {
    if (k <= 0 || k % 16 || m < 0 || (m && k > (int64_t(1) << 40) / m)) return TQ2_ERR_INVALID_ARG;
    if (m == 0) return TQ2_OK;
    if (!x || !x16) return TQ2_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(x16)) return TQ2_ERR_MISALIGNED;
    if (overlaps(x, size_t(m) * size_t(k) * 4, x16, size_t(m) * size_t(k) * 2)) return TQ2_ERR_INVALID_ARG;
    tq2::LaunchCtx ctx;
    int st = prepare(stream, &ctx, {x, x16});
    if (st != TQ2_OK) return st;
    return finish(tq2::launch_act16_from_f32(x, static_cast<__half *>(x16), m, k, ctx));
}

int tq2_act16_to_f32(const void *x16, float *x, int64_t m, int64_t k, void *stream) {
    if (k <= 0 || k % 16 || m < 0 || (m && k > (int64_t(1) << 40) / m)) return TQ2_ERR_INVALID_ARG;
    if (m == 0) return TQ2_OK;
    if (!x || !x16) return TQ2_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(x16)) return TQ2_ERR_MISALIGNED;
    if (overlaps(x, size_t(m) * size_t(k) * 4, x16, size_t(m) * size_t(k) * 2)) return TQ2_ERR_INVALID_ARG;
    tq2::LaunchCtx ctx;
    int st = prepare(stream, &ctx, {x16, x});
    if (st != TQ2_OK) return st;
    return finish(tq2::launch_act16_to_f32(static_cast<const __half *>(x16), x, m, k, ctx));
}

int tq2_gemm_act16(const void *w_soa, const void *x16, const void *residual16, void *out16, int64_t m,
                   int64_t n, int64_t k, void *stream) {
    bool noop = false;
    int st = check_shape(m, n, k, &noop);
    if (st != TQ2_OK || noop) return st;
    if (n % 16) return TQ2_ERR_INVALID_ARG;
    if (!w_soa || !x16 || !out16) return TQ2_ERR_INVALID_ARG;
    if (!aligned16(w_soa) || !aligned16(x16) || !aligned16(out16) || (residual16 && !aligned16(residual16)))
        return TQ2_ERR_MISALIGNED;
    const size_t wb = size_t(n) * size_t(k / tq2::kBlockW) * tq2::kBlockBytes;
    const size_t xb = size_t(m) * size_t(k) * 2, ob = size_t(m) * size_t(n) * 2;
    if (overlaps(out16, ob, x16, xb) || overlaps(out16, ob, w_soa, wb)) return TQ2_ERR_INVALID_ARG;
    if (residual16 && residual16 != out16 && overlaps(out16, ob, residual16, ob)) return TQ2_ERR_INVALID_ARG;
    tq2::LaunchCtx ctx;
    st = prepare(stream, &ctx, {w_soa, x16, residual16, out16});
    if (st != TQ2_OK) return st;
    const size_t need = tq2::tc_act16_ws_bytes(m, n, k);
    void *ws = nullptr;
    if (need && cudaMallocAsync(&ws, need, ctx.stream) != cudaSuccess) {
        (void)cudaGetLastError();
        return TQ2_ERR_CUDA;
    }
    cudaError_t e = tq2::launch_tc_act16(w_soa, static_cast<const __half *>(x16),
                                         static_cast<const __half *>(residual16), static_cast<__half *>(out16),
                                         m, n, k, ws, ctx);
    if (ws) {
        const cudaError_t f = cudaFreeAsync(ws, ctx.stream);
        if (e == cudaSuccess) e = f;
    }
    return finish(e);
}

int tq2_attention_f32(const float *q, const float *k, const float *v, float *out, int64_t heads,
                      int64_t seq, int64_t dim, void *stream) {
    if (heads < 0 || seq < 0 || dim < 8 || dim > 128 || dim % 8) return TQ2_ERR_INVALID_ARG;
    if (heads > 65535 || seq > (int64_t(1) << 24) || heads * ((seq + 127) / 128 * 128) > INT32_MAX)
        return TQ2_ERR_INVALID_ARG;
    if (heads == 0 || seq == 0) return TQ2_OK;
    if (!q || !k || !v || !out) return TQ2_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out)) return TQ2_ERR_MISALIGNED;
    const size_t nb = size_t(heads) * size_t(seq) * size_t(dim) * 4;
    if (overlaps(out, nb, q, nb) || overlaps(out, nb, k, nb) || overlaps(out, nb, v, nb))
        return TQ2_ERR_INVALID_ARG;
    tq2::LaunchCtx ctx;
    int st = prepare(stream, &ctx, {q, k, v, out});
    if (st != TQ2_OK) return st;
    void *ws = nullptr;
    if (cudaMallocAsync(&ws, tq2::attention_ws_bytes(heads, seq, dim), ctx.stream) != cudaSuccess) {
        (void)cudaGetLastError();
        return TQ2_ERR_CUDA;
    }
    cudaError_t e = tq2::launch_attention(q, k, v, out, heads, seq, dim, ws, ctx);
    const cudaError_t f = cudaFreeAsync(ws, ctx.stream);
    return finish(e != cudaSuccess ? e : f);
}

int tq2_gemv(const void *w_soa, const float *x, const float *residual, float *out, int64_t n,
             int64_t k, void *stream) {
    return tq2_gemm_with(TQ2_KERNEL_GEMV, w_soa, x, residual, out, 1, n, k, stream);
}

int tq2_gemv_resident(const void *w_soa, const float *x, const float *residual, float *out,
                      int64_t n, int64_t k, void *stream) {
    bool noop = false;
    int st = check_matmul(w_soa, x, residual, out, 1, n, k, &noop);
    if (st != TQ2_OK || noop) return st;
    tq2::LaunchCtx ctx;
    st = prepare(stream, &ctx, {w_soa, x, residual, out});
    if (st != TQ2_OK) return st;
    return finish(tq2::launch_gemv(w_soa, x, residual, out, n, k, ctx, true));
}

int tq2_gemm_f32ref(const void *w_soa, const float *x, const float *residual, float *out,
                    int64_t m, int64_t n, int64_t k, void *stream) {
    return tq2_gemm_with(TQ2_KERNEL_F32REF, w_soa, x, residual, out, m, n, k, stream);
}

// ---------------------------------------------------------------------------
// positions, key/value cache and its attention

namespace {

constexpr int64_t kMaxHeads = 16384;
constexpr int64_t kMaxTokens = int64_t(1) << 30;
constexpr int64_t kMaxStride = int64_t(1) << 40;

size_t dtype_bytes(int dtype) { return dtype == TQ2_F32 ? 4 : 2; }
bool dtype_ok(int dtype) { return dtype == TQ2_F32 || dtype == TQ2_F16 || dtype == TQ2_BF16; }

// The elements of a view whose innermost `dim` are contiguous are distinct: with
// the strides in order, each steps over all that lies below it.
bool distinct(int64_t dim, int64_t n0, int64_t s0, int64_t n1, int64_t s1) {
    if (n0 == 1) return n1 == 1 || s1 >= dim;
    if (n1 == 1) return s0 >= dim;
    if (s0 > s1) return s1 >= dim && s0 >= (n1 - 1) * s1 + dim;
    return s0 >= dim && s1 >= (n0 - 1) * s0 + dim;
}

int check_view(const tq2_heads *v, int64_t tokens, int64_t dim, bool output) {
    if (!v->data || !dtype_ok(v->dtype)) return TQ2_ERR_INVALID_ARG;
    if (v->heads < 1 || v->heads > kMaxHeads || v->token_stride < 0 || v->head_stride < 0 ||
        v->token_stride > kMaxStride || v->head_stride > kMaxStride ||
        (v->token_stride && tokens > (int64_t(1) << 44) / v->token_stride))
        return TQ2_ERR_INVALID_ARG;
    if (output && !distinct(dim, tokens, v->token_stride, v->heads, v->head_stride)) return TQ2_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(v->data) % dtype_bytes(v->dtype)) return TQ2_ERR_MISALIGNED;
    return TQ2_OK;
}

// A stride along an axis of one element says nothing: such strides become 0.
tq2_heads plain_view(const tq2_heads *v, int64_t tokens) {
    tq2_heads r = *v;
    if (tokens == 1) r.token_stride = 0;
    if (r.heads == 1) r.head_stride = 0;
    return r;
}
tq2_kv_cache plain_cache(const tq2_kv_cache *c) {
    tq2_kv_cache r = *c;
    if (r.pages == 1) r.page_stride = 0;
    if (r.page_size == 1) r.slot_stride = 0;
    if (r.heads == 1) r.head_stride = 0;
    return r;
}

bool same_view(const tq2_heads *a, const tq2_heads *b) {
    return a->data == b->data && a->dtype == b->dtype && a->heads == b->heads &&
           a->token_stride == b->token_stride && a->head_stride == b->head_stride;
}

// Whether two views share no byte: their extents lie apart, or they are different columns of rows with one stride
// (slices of one fused projection), or, stepping alike, no piece of one head meets one of the other (q, k and v
// interleaved by head).  Views that mesh with strides of their own count as overlapping.
bool views_apart(const tq2_heads *a, const tq2_heads *b, int64_t tokens, int64_t dim) {
    const size_t ea = dtype_bytes(a->dtype), eb = dtype_bytes(b->dtype);
    const size_t wa = size_t((a->heads - 1) * a->head_stride + dim) * ea;
    const size_t wb = size_t((b->heads - 1) * b->head_stride + dim) * eb;
    const size_t ra = size_t(a->token_stride) * ea, rb = size_t(b->token_stride) * eb;
    if (!overlaps(a->data, size_t(tokens - 1) * ra + wa, b->data, size_t(tokens - 1) * rb + wb)) return true;
    if (ra != rb) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a->data), y = reinterpret_cast<uintptr_t>(b->data);
    if (wa <= ra && wb <= ra) {
        const size_t d = y >= x ? (y - x) % ra : (ra - (x - y) % ra) % ra;  // b's columns, from a's first
        if (d >= wa && d + wb <= ra) return true;
    }
    const int64_t sa = a->head_stride * int64_t(ea), sb = b->head_stride * int64_t(eb);
    if (a->heads > 1 && b->heads > 1 && sa != sb) return false;
    const int64_t pa = dim * int64_t(ea), pb = dim * int64_t(eb), s = a->heads > 1 ? sa : sb, r = int64_t(ra);
    // a piece of b starts at (its head - a's head) * s + (its token - a's token) * r + y - x from one of a: within -pb and pa
    // they meet
    const int64_t base = y >= x ? int64_t(y - x) : -int64_t(x - y);
    auto floor_div = [](int64_t n, int64_t d) { return n / d - (n % d < 0); };
    for (int64_t h = 1 - a->heads; h < b->heads; ++h) {
        const int64_t at = base + h * s;
        if (r == 0) {
            if (at > -pb && at < pa) return false;
        } else {
            const int64_t lo = floor_div(-pb - at, r) + 1, hi = floor_div(pa - 1 - at, r);  // token differences that meet
            if (lo <= hi && lo < tokens && hi > -tokens) return false;
        }
    }
    return true;
}

// bytes from the first to the last element of a cache plane
size_t plane_bytes(const tq2_kv_cache *c) {
    return size_t((c->pages - 1) * c->page_stride + (c->page_size - 1) * c->slot_stride +
                  (c->heads - 1) * c->head_stride + c->dim) * 2;
}

bool view_in_plane(const tq2_heads *v, int64_t tokens, const tq2_kv_cache *c, const void *plane) {
    const size_t n = size_t((tokens - 1) * v->token_stride + (v->heads - 1) * v->head_stride + c->dim) *
                     dtype_bytes(v->dtype);
    return overlaps(v->data, n, plane, plane_bytes(c));
}

int check_cache(const tq2_kv_cache *c) {
    if (!c->k || !c->v || (c->dtype != TQ2_F16 && c->dtype != TQ2_BF16)) return TQ2_ERR_INVALID_ARG;
    if (c->dim < 8 || c->dim > 128 || c->dim % 8 || c->heads < 1 || c->heads > kMaxHeads) return TQ2_ERR_INVALID_ARG;
    if (c->pages < 1 || c->pages > INT32_MAX || c->page_size < 1 || c->page_size > (1 << 20)) return TQ2_ERR_INVALID_ARG;
    int64_t n[3] = {c->pages, c->page_size, c->heads}, s[3] = {c->page_stride, c->slot_stride, c->head_stride};
    for (int i = 0; i < 3; ++i)
        if (s[i] < 0 || s[i] > kMaxStride / 8 || (s[i] && n[i] > (int64_t(1) << 44) / s[i])) return TQ2_ERR_INVALID_ARG;
    for (int i = 0; i < 3; ++i)  // ascending strides
        for (int j = i + 1; j < 3; ++j)
            if (s[j] < s[i]) {
                const int64_t tn = n[i], ts = s[i];
                n[i] = n[j], s[i] = s[j], n[j] = tn, s[j] = ts;
            }
    int64_t below = c->dim;
    for (int i = 0; i < 3; ++i) {
        if (n[i] == 1) continue;
        if (s[i] < below) return TQ2_ERR_INVALID_ARG;
        below += (n[i] - 1) * s[i];
    }
    if (!aligned16(c->k) || !aligned16(c->v) || c->page_stride % 8 || c->slot_stride % 8 || c->head_stride % 8)
        return TQ2_ERR_MISALIGNED;
    return TQ2_OK;
}

// shape checks of a batch (its pointers are looked at only where there is work)
int check_batch_shape(const tq2_batch *b, bool *noop) {
    *noop = false;
    if (!b || b->seqs < 0 || b->seqs > (1 << 20) || b->tokens < 0 || b->tokens > kMaxTokens || b->max_q < 0 ||
        b->max_q > kMaxTokens || b->max_kv < 0 || b->max_kv > kMaxTokens || b->table_stride < 0 ||
        b->table_stride > INT32_MAX)
        return TQ2_ERR_INVALID_ARG;
    if (b->seqs == 0 || b->tokens == 0 || b->max_q == 0) *noop = true;
    return TQ2_OK;
}

int check_batch(const tq2_batch *b) {
    if (!b->q_start || !b->kv_len || (!b->page_table && b->table_stride)) return TQ2_ERR_INVALID_ARG;
    for (const int32_t *p : {b->q_start, b->kv_len, b->page_table})
        if (reinterpret_cast<uintptr_t>(p) % 4) return TQ2_ERR_MISALIGNED;
    return TQ2_OK;
}

tq2::BatchView batch_view(const tq2_batch *b, const tq2_kv_cache *c) {
    tq2::BatchView v = {};
    v.q_start = b->q_start;
    v.kv_len = b->kv_len;
    v.page_table = b->page_table;
    v.tokens = b->tokens;
    v.table_stride = b->table_stride;
    v.pages = c->pages;
    v.seqs = int(b->seqs);
    v.max_q = int(b->max_q < b->tokens ? b->max_q : b->tokens);
    const int64_t width = b->table_stride * c->page_size;  // (a loose max_kv sizes nothing beyond the table)
    v.max_kv = int(b->max_kv < width ? b->max_kv : width);
    v.page_size = int(c->page_size);
    return v;
}

// rope may be NULL (no rotation); positions_needed: NULL positions are refused
int check_rope(const tq2_rope *r, const int64_t *positions, int64_t dim, bool positions_needed) {
    if (!r) return TQ2_OK;
    if (r->pairs < 0 || 2 * r->pairs > dim || r->axes < 1 || r->axes > 16) return TQ2_ERR_INVALID_ARG;
    if (r->pairs == 0) return TQ2_OK;
    if (!r->turns || (!positions && (positions_needed || r->axes != 1))) return TQ2_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(r->turns) % 8 || reinterpret_cast<uintptr_t>(positions) % 8)
        return TQ2_ERR_MISALIGNED;
    return TQ2_OK;
}

void set_rope(tq2::RopeArgs *a, const tq2_rope *r, const int64_t *positions, int64_t dim) {
    a->dim = int(dim);
    a->axes = 1;
    if (!r) return;
    a->positions = positions;
    a->turns = r->turns;
    a->axis = r->axis;
    a->axes = r->axes;
    a->pairs = int(r->pairs);
    a->interleaved = r->interleaved != 0;
}

void add_segment(tq2::RopeArgs *a, const tq2_heads *in, const tq2_heads *out, bool turned) {
    tq2::RopeSegment &g = a->seg[a->nseg++];
    g.in = in->data;
    g.in_token = in->token_stride;
    g.in_head = in->head_stride;
    g.heads = int(in->heads);
    g.turned = turned;
    if (out) {
        g.out = out->data;
        g.out_token = out->token_stride;
        g.out_head = out->head_stride;
    }
}

}  // namespace

int tq2_rope_turns(const double *inv_freq, uint64_t *turns, int64_t pairs) {
    if (pairs < 0 || (pairs && (!inv_freq || !turns))) return TQ2_ERR_INVALID_ARG;
    for (int64_t i = 0; i < pairs; ++i)
        if (!std::isfinite(inv_freq[i])) return TQ2_ERR_INVALID_ARG;
    for (int64_t i = 0; i < pairs; ++i) {
        const double t = inv_freq[i] / 6.283185307179586476925286766559;
        const double f = std::fmod(std::fabs(t), 1.0);  // [0, 1), exact
        // 2^64 f in two halves (the upper one exact), negated as an integer
        const double hi = std::floor(f * 0x1p32);
        const uint64_t u = (uint64_t(hi) << 32) + uint64_t(std::llrint((f * 0x1p32 - hi) * 0x1p32));
        turns[i] = t < 0 ? 0 - u : u;
    }
    return TQ2_OK;
}

int tq2_rope_axes(const tq2_heads *q, const tq2_heads *q_out, const tq2_heads *k, const tq2_heads *k_out,
                  const tq2_heads *v, const tq2_heads *v_out, const int64_t *positions, const tq2_rope *rope,
                  int64_t tokens, int64_t dim, int inverse, void *stream) {
    if (tokens < 0 || tokens > kMaxTokens || dim < 1 || dim > 65536 || !rope) return TQ2_ERR_INVALID_ARG;
    if (rope->pairs < 0 || 2 * rope->pairs > dim || rope->axes < 1 || rope->axes > 16) return TQ2_ERR_INVALID_ARG;
    if (tokens == 0) return TQ2_OK;
    if (!q || !q_out || !k != !k_out || !v != !v_out) return TQ2_ERR_INVALID_ARG;
    int st = check_rope(rope, positions, dim, true);
    if (st != TQ2_OK) return st;
    tq2_heads plain[6];
    const tq2_heads *in[3] = {q, k, v}, *out[3] = {q_out, k_out, v_out};
    for (int i = 0; i < 3; ++i) {
        if (!in[i]) continue;
        plain[i] = plain_view(in[i], tokens);
        plain[3 + i] = plain_view(out[i], tokens);
        in[i] = &plain[i];
        out[i] = &plain[3 + i];
        if ((st = check_view(in[i], tokens, dim, false)) != TQ2_OK) return st;
        if ((st = check_view(out[i], tokens, dim, true)) != TQ2_OK) return st;
        if (in[i]->heads != out[i]->heads || in[i]->dtype != q->dtype || out[i]->dtype != q_out->dtype)
            return TQ2_ERR_INVALID_ARG;
    }
    for (int i = 0; i < 3; ++i)
        for (int j = 0; j < 3; ++j) {
            if (!in[i] || !in[j]) continue;
            if (!(i == j && same_view(out[i], in[j])) && !views_apart(out[i], in[j], tokens, dim))
                return TQ2_ERR_INVALID_ARG;
            if (i < j && !views_apart(out[i], out[j], tokens, dim)) return TQ2_ERR_INVALID_ARG;
        }
    tq2::LaunchCtx ctx;
    st = prepare(stream, &ctx, {q->data, q_out->data, k ? k->data : nullptr, k ? k_out->data : nullptr,
                                v ? v->data : nullptr, v ? v_out->data : nullptr,
                                rope->pairs ? positions : nullptr, rope->pairs ? rope->turns : nullptr,
                                rope->pairs ? rope->axis : nullptr});
    if (st != TQ2_OK) return st;
    tq2::RopeArgs a = {};
    set_rope(&a, rope, positions, dim);
    a.tokens = tokens;
    a.inverse = inverse != 0;
    for (int i = 0; i < 3; ++i)
        if (in[i]) add_segment(&a, in[i], out[i], i < 2);
    return finish(tq2::launch_rope(a, q->dtype, q_out->dtype, ctx));
}

int tq2_kv_append(const tq2_heads *q, const tq2_heads *q_out, const tq2_heads *k, const tq2_heads *v,
                  const int64_t *positions, const tq2_rope *rope, const tq2_batch *batch, const tq2_kv_cache *cache,
                  void *stream) {
    bool noop = false;
    int st = check_batch_shape(batch, &noop);
    if (st != TQ2_OK) return st;
    if (!cache) return TQ2_ERR_INVALID_ARG;
    const tq2_kv_cache cv = plain_cache(cache);
    cache = &cv;
    if ((st = check_cache(cache)) != TQ2_OK) return st;
    if ((st = check_rope(rope, positions, cache->dim, false)) != TQ2_OK) return st;
    if (noop) return TQ2_OK;
    if ((st = check_batch(batch)) != TQ2_OK) return st;
    if (!k || !v || !q != !q_out) return TQ2_ERR_INVALID_ARG;
    const int64_t tokens = batch->tokens, dim = cache->dim;
    tq2_heads plain[4];
    int np = 0;
    for (const tq2_heads **x : {&q, &q_out, &k, &v})
        if (*x) {
            plain[np] = plain_view(*x, tokens);
            *x = &plain[np++];
        }
    if ((st = check_view(k, tokens, dim, false)) != TQ2_OK || (st = check_view(v, tokens, dim, false)) != TQ2_OK)
        return st;
    if (k->heads != cache->heads || v->heads != cache->heads || k->dtype != v->dtype) return TQ2_ERR_INVALID_ARG;
    if (q) {
        if ((st = check_view(q, tokens, dim, false)) != TQ2_OK || (st = check_view(q_out, tokens, dim, true)) != TQ2_OK)
            return st;
        if (q->heads != q_out->heads || q->dtype != k->dtype || q_out->dtype != cache->dtype) return TQ2_ERR_INVALID_ARG;
        if (!same_view(q, q_out) && !views_apart(q, q_out, tokens, dim)) return TQ2_ERR_INVALID_ARG;
        if (!views_apart(q_out, k, tokens, dim) || !views_apart(q_out, v, tokens, dim)) return TQ2_ERR_INVALID_ARG;
    }
    for (const tq2_heads *x : {q, q_out, k, v})
        if (x && (view_in_plane(x, tokens, cache, cache->k) || view_in_plane(x, tokens, cache, cache->v)))
            return TQ2_ERR_INVALID_ARG;
    tq2::LaunchCtx ctx;
    const bool turns = rope && rope->pairs;
    st = prepare(stream, &ctx, {q ? q->data : nullptr, q ? q_out->data : nullptr, k->data, v->data,
                                turns ? positions : nullptr, turns ? rope->turns : nullptr,
                                turns ? rope->axis : nullptr, batch->q_start, batch->kv_len, batch->page_table,
                                cache->k, cache->v});
    if (st != TQ2_OK) return st;
    tq2::RopeArgs a = {};
    set_rope(&a, rope, positions, dim);
    a.tokens = tokens;
    a.append = 1;
    a.batch = batch_view(batch, cache);
    a.page_stride = cache->page_stride;
    if (q) add_segment(&a, q, q_out, true);
    for (int i = 0; i < 2; ++i) {
        add_segment(&a, i ? v : k, nullptr, i == 0);
        tq2::RopeSegment &g = a.seg[a.nseg - 1];
        g.out = i ? cache->v : cache->k;
        g.out_token = cache->slot_stride;
        g.out_head = cache->head_stride;
        g.paged = 1;
    }
    return finish(tq2::launch_rope(a, k->dtype, cache->dtype, ctx));
}

size_t tq2_attention_paged_workspace_bytes(int64_t heads, const tq2_kv_cache *cache, const tq2_batch *batch) {
    bool noop = false;
    if (check_batch_shape(batch, &noop) != TQ2_OK || noop || !cache || cache->heads < 1 || cache->heads > kMaxHeads ||
        heads < 1 || heads > kMaxHeads || heads % cache->heads || cache->dim < 8 || cache->dim > 128 || cache->dim % 8)
        return 0;
    return tq2::attention_paged_ws_bytes(heads, cache->heads, cache->dim, batch->seqs, batch->tokens, batch->max_q,
                                         batch->max_kv);
}

int tq2_attention_paged(const tq2_heads *q, const tq2_heads *out, const tq2_kv_cache *cache, const tq2_batch *batch,
                        float scale, int64_t window, int causal, void *workspace, size_t workspace_bytes,
                        void *stream) {
    bool noop = false;
    int st = check_batch_shape(batch, &noop);
    if (st != TQ2_OK) return st;
    if (!cache) return TQ2_ERR_INVALID_ARG;
    const tq2_kv_cache cv = plain_cache(cache);
    cache = &cv;
    if ((st = check_cache(cache)) != TQ2_OK) return st;
    if (!std::isfinite(scale) || window < 0) return TQ2_ERR_INVALID_ARG;
    if (noop) return TQ2_OK;
    if ((st = check_batch(batch)) != TQ2_OK) return st;
    if (!q || !out) return TQ2_ERR_INVALID_ARG;
    const int64_t tokens = batch->tokens, dim = cache->dim;
    const tq2_heads qv = plain_view(q, tokens), ov = plain_view(out, tokens);
    q = &qv;
    out = &ov;
    if ((st = check_view(q, tokens, dim, false)) != TQ2_OK || (st = check_view(out, tokens, dim, true)) != TQ2_OK)
        return st;
    if (q->heads != out->heads || q->heads % cache->heads || q->dtype != cache->dtype ||
        (out->dtype != cache->dtype && out->dtype != TQ2_F32) || tokens * (q->heads / cache->heads) > INT32_MAX - 1024)
        return TQ2_ERR_INVALID_ARG;
    for (const tq2_heads *x : {q, out})
        if (!aligned16(x->data) || x->token_stride % 8 || x->head_stride % 8) return TQ2_ERR_MISALIGNED;
    if (!views_apart(q, out, tokens, dim) || view_in_plane(out, tokens, cache, cache->k) ||
        view_in_plane(out, tokens, cache, cache->v))
        return TQ2_ERR_INVALID_ARG;
    const size_t need = tq2_attention_paged_workspace_bytes(q->heads, cache, batch);
    if (workspace) {
        if (workspace_bytes < need) return TQ2_ERR_INVALID_ARG;
        if (!aligned16(workspace)) return TQ2_ERR_MISALIGNED;
        const size_t nb = size_t((tokens - 1) * q->token_stride + (q->heads - 1) * q->head_stride + dim) * 2;
        const size_t ob = size_t((tokens - 1) * out->token_stride + (out->heads - 1) * out->head_stride + dim) *
                          dtype_bytes(out->dtype);
        if (overlaps(workspace, need, q->data, nb) || overlaps(workspace, need, out->data, ob) ||
            overlaps(workspace, need, cache->k, plane_bytes(cache)) ||
            overlaps(workspace, need, cache->v, plane_bytes(cache)))
            return TQ2_ERR_INVALID_ARG;
    }
    tq2::LaunchCtx ctx;
    st = prepare(stream, &ctx, {q->data, out->data, cache->k, cache->v, batch->q_start, batch->kv_len,
                                batch->page_table, workspace});
    if (st != TQ2_OK) return st;
    tq2::PagedArgs a = {};
    a.q = q->data;
    a.out = out->data;
    a.k = cache->k;
    a.v = cache->v;
    a.q_token = q->token_stride;
    a.q_head = q->head_stride;
    a.out_token = out->token_stride;
    a.out_head = out->head_stride;
    a.page_stride = cache->page_stride;
    a.slot_stride = cache->slot_stride;
    a.head_stride = cache->head_stride;
    a.batch = batch_view(batch, cache);
    a.window = window;
    a.scale = scale;
    a.heads = int(q->heads);
    a.kv_heads = int(cache->heads);
    a.dim = int(dim);
    a.causal = causal != 0;
    void *ws = workspace;
    if (need && !ws && cudaMallocAsync(&ws, need, ctx.stream) != cudaSuccess) {
        (void)cudaGetLastError();
        return TQ2_ERR_CUDA;
    }
    const cudaError_t e = tq2::launch_attention_paged(a, cache->dtype, out->dtype == TQ2_F32, ws, ctx);
    const cudaError_t f = ws != workspace ? cudaFreeAsync(ws, ctx.stream) : cudaSuccess;
    return finish(e != cudaSuccess ? e : f);
}

// ---------------------------------------------------------------------------
// mixtures of experts, sampling

namespace {

constexpr int64_t kMaxExperts = 1024, kMaxTopK = 32, kMaxFeatures = 65536, kMaxPairs = int64_t(1) << 22;
constexpr int64_t kMaxVocabulary = int64_t(1) << 18, kMaxRows = int64_t(1) << 24;

// Rows of logits: [rows, n], row r from element r * stride on.
int check_logits(const void *logits, int dtype, int64_t stride, int64_t rows, int64_t n) {
    if (!logits || !dtype_ok(dtype)) return TQ2_ERR_INVALID_ARG;
    if (rows > 1 && (stride < n || stride > kMaxStride)) return TQ2_ERR_INVALID_ARG;
    return reinterpret_cast<uintptr_t>(logits) % dtype_bytes(dtype) ? TQ2_ERR_MISALIGNED : TQ2_OK;
}
size_t logits_bytes(int dtype, int64_t stride, int64_t rows, int64_t n) {
    return size_t((rows - 1) * (rows > 1 ? stride : 0) + n) * dtype_bytes(dtype);
}

bool misaligned(const void *p, size_t to) { return reinterpret_cast<uintptr_t>(p) % to != 0; }

int check_experts(const tq2_experts *w, int dtype, int64_t tokens, int64_t top_k) {
    if (!w || !dtype_ok(dtype)) return TQ2_ERR_INVALID_ARG;
    if (w->width <= 0 || w->width % tq2::kBlockW || w->ffn <= 0 || w->ffn % tq2::kBlockW) return TQ2_ERR_BAD_K;
    if (w->width > kMaxFeatures || w->ffn > kMaxFeatures || w->experts < 1 || w->experts > kMaxExperts || top_k < 1 ||
        top_k > kMaxTopK || tokens < 0 || tokens > kMaxPairs / top_k)
        return TQ2_ERR_INVALID_ARG;
    // rows of a weight are counted in 32 bits
    if (w->experts * 2 * w->ffn > INT32_MAX || w->experts * w->width > INT32_MAX) return TQ2_ERR_INVALID_ARG;
    return TQ2_OK;
}

}  // namespace

int tq2_moe_route(const void *logits, int dtype, int64_t row_stride, int32_t *experts, float *weights, int64_t tokens,
                  int64_t n_experts, int64_t top_k, int sigmoid, int normalize, float scale, void *stream) {
    if (tokens < 0 || tokens > kMaxRows || n_experts < 1 || n_experts > kMaxExperts || top_k < 1 || top_k > kMaxTopK ||
        top_k > n_experts || !std::isfinite(scale) || !dtype_ok(dtype))
        return TQ2_ERR_INVALID_ARG;
    if (tokens == 0) return TQ2_OK;
    int st = check_logits(logits, dtype, row_stride, tokens, n_experts);
    if (st != TQ2_OK) return st;
    if (!experts || !weights) return TQ2_ERR_INVALID_ARG;
    if (misaligned(experts, 4) || misaligned(weights, 4)) return TQ2_ERR_MISALIGNED;
    const size_t lb = logits_bytes(dtype, row_stride, tokens, n_experts), ob = size_t(tokens) * size_t(top_k) * 4;
    if (overlaps(experts, ob, logits, lb) || overlaps(weights, ob, logits, lb) || overlaps(experts, ob, weights, ob))
        return TQ2_ERR_INVALID_ARG;
    tq2::LaunchCtx ctx;
    st = prepare(stream, &ctx, {logits, experts, weights});
    if (st != TQ2_OK) return st;
    tq2::RouteArgs a = {};
    a.logits = logits;
    a.row_stride = tokens > 1 ? row_stride : 0;
    a.experts = experts;
    a.weights = weights;
    a.tokens = tokens;
    a.n = int(n_experts);
    a.top_k = int(top_k);
    a.sigmoid = sigmoid != 0;
    a.normalize = normalize != 0;
    a.scale = scale;
    return finish(tq2::launch_moe_route(a, dtype, ctx));
}

size_t tq2_moe_swiglu_workspace_bytes(const tq2_experts *w, int dtype, int64_t tokens, int64_t top_k) {
    if (check_experts(w, dtype, tokens, top_k) != TQ2_OK || tokens == 0) return 0;
    return tq2::moe_ws_bytes(tokens, top_k, w->experts, w->width, w->ffn, dtype);
}

int tq2_moe_swiglu(const tq2_experts *w, const void *x, const int32_t *expert, const float *weight,
                   const void *residual, void *out, int dtype, int64_t tokens, int64_t top_k, void *workspace,
                   size_t workspace_bytes, void *stream) {
    int st = check_experts(w, dtype, tokens, top_k);
    if (st != TQ2_OK || tokens == 0) return st;
    if (!w->gate_up || !w->down || !x || !expert || !weight || !out) return TQ2_ERR_INVALID_ARG;
    if (!aligned16(w->gate_up) || !aligned16(w->down) || !aligned16(x) || !aligned16(out) ||
        (residual && !aligned16(residual)) || misaligned(expert, 4) || misaligned(weight, 4))
        return TQ2_ERR_MISALIGNED;
    const size_t xb = size_t(tokens) * size_t(w->width) * dtype_bytes(dtype), pb = size_t(tokens) * size_t(top_k) * 4;
    const size_t gb = tq2_soa_bytes(w->experts * 2 * w->ffn, w->width), db = tq2_soa_bytes(w->experts * w->width, w->ffn);
    const size_t need = tq2::moe_ws_bytes(tokens, top_k, w->experts, w->width, w->ffn, dtype);
    if (workspace && workspace_bytes < need) return TQ2_ERR_INVALID_ARG;
    if (workspace && !aligned16(workspace)) return TQ2_ERR_MISALIGNED;
    const struct {
        const void *p;
        size_t n;
    } in[] = {{x, xb}, {expert, pb}, {weight, pb}, {w->gate_up, gb}, {w->down, db}, {residual, residual ? xb : 0}};
    for (const auto &i : in)
        if ((i.p != residual || residual != out) && overlaps(out, xb, i.p, i.n)) return TQ2_ERR_INVALID_ARG;
    if (workspace) {
        if (overlaps(workspace, need, out, xb)) return TQ2_ERR_INVALID_ARG;
        for (const auto &i : in)
            if (overlaps(workspace, need, i.p, i.n)) return TQ2_ERR_INVALID_ARG;
    }
    tq2::LaunchCtx ctx;
    st = prepare(stream, &ctx, {w->gate_up, w->down, x, expert, weight, residual, out, workspace});
    if (st != TQ2_OK) return st;
    tq2::MoeArgs a = {};
    a.gate_up = w->gate_up;
    a.down = w->down;
    a.x = x;
    a.residual = residual;
    a.expert = expert;
    a.weight = weight;
    a.out = out;
    a.tokens = tokens;
    a.experts = int(w->experts);
    a.width = int(w->width);
    a.ffn = int(w->ffn);
    a.top_k = int(top_k);
    void *ws = workspace;
    if (!ws && cudaMallocAsync(&ws, need, ctx.stream) != cudaSuccess) {
        (void)cudaGetLastError();
        return TQ2_ERR_CUDA;
    }
    const cudaError_t e = tq2::launch_moe(a, dtype, ws, ctx);
    const cudaError_t f = ws != workspace ? cudaFreeAsync(ws, ctx.stream) : cudaSuccess;
    return finish(e != cudaSuccess ? e : f);
}

int tq2_sample(const void *logits, int dtype, int64_t row_stride, const float *u, const tq2_sampling *filters,
               int64_t *tokens, float *prob, int64_t rows, int64_t vocab, void *stream) {
    if (rows < 0 || rows > kMaxRows || vocab < 1 || vocab > kMaxVocabulary || !dtype_ok(dtype)) return TQ2_ERR_INVALID_ARG;
    if (rows == 0) return TQ2_OK;
    int st = check_logits(logits, dtype, row_stride, rows, vocab);
    if (st != TQ2_OK) return st;
    if (!u || !tokens) return TQ2_ERR_INVALID_ARG;
    const tq2_sampling off = {};
    const tq2_sampling f = filters ? *filters : off;
    const void *in[] = {u, f.temperature, f.top_k, f.top_p, f.min_p};
    if (misaligned(tokens, 8) || misaligned(prob, 4)) return TQ2_ERR_MISALIGNED;
    for (const void *p : in)
        if (misaligned(p, 4)) return TQ2_ERR_MISALIGNED;
    const size_t lb = logits_bytes(dtype, row_stride, rows, vocab), rb = size_t(rows) * 4;
    if (overlaps(tokens, 2 * rb, logits, lb)) return TQ2_ERR_INVALID_ARG;
    if (prob && (overlaps(prob, rb, logits, lb) || overlaps(prob, rb, tokens, 2 * rb))) return TQ2_ERR_INVALID_ARG;
    for (const void *p : in)
        if (p && (overlaps(tokens, 2 * rb, p, rb) || (prob && overlaps(prob, rb, p, rb)))) return TQ2_ERR_INVALID_ARG;
    tq2::LaunchCtx ctx;
    st = prepare(stream, &ctx, {logits, u, f.temperature, f.top_k, f.top_p, f.min_p, tokens, prob});
    if (st != TQ2_OK) return st;
    tq2::SampleArgs a = {};
    a.logits = logits;
    a.row_stride = rows > 1 ? row_stride : 0;
    a.u = u;
    a.temperature = f.temperature;
    a.top_k = f.top_k;
    a.top_p = f.top_p;
    a.min_p = f.min_p;
    a.tokens = tokens;
    a.prob = prob;
    a.rows = rows;
    a.vocab = int(vocab);
    return finish(tq2::launch_sample(a, dtype, ctx));
}

}  // extern "C"
