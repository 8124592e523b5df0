"""Python binding of the GB300 TQ2_0_g128 ternary matmul library.

Argument marshalling only: every entry point forwards raw device pointers,
sizes and a CUDA stream to the C ABI declared in ``include/tq2.h`` (loaded
from ``libtq2_gb300.so`` next to this file) and turns a non-zero status into
``TQ2Error``.  All arithmetic runs in the library's CUDA kernels; there is no
Python or CPU fallback, and importing this package fails loudly when the
library has not been built.

Arguments that take device memory accept a torch CUDA tensor or a raw integer
pointer.  ``stream`` accepts a ``torch.cuda.Stream``, a raw ``cudaStream_t``
integer, or None (the current torch stream when torch is importable, else the
legacy default stream).
"""

from __future__ import annotations

import contextlib
import ctypes
import os
import struct

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libtq2_gb300.so")

TQ2_OK = 0
TQ2_ERR_INVALID_ARG = 1
TQ2_ERR_BAD_K = 2
TQ2_ERR_MISALIGNED = 3
TQ2_ERR_UNSUPPORTED_DEVICE = 4
TQ2_ERR_CUDA = 5
TQ2_ERR_TIMEOUT = 6
TQ2_ERR_TOO_LARGE = 7
TQ2_ERR_BAD_BATCH = 8
TQ2_NOALLOC_SCRATCH_BYTES = 32 * 1024 * 1024

TQ2_KERNEL_AUTO = 0
TQ2_KERNEL_GEMV = 1
TQ2_KERNEL_SKINNY = 2
TQ2_KERNEL_TC = 3
TQ2_KERNEL_F32REF = 4
TQ2_KERNEL_TC_DIRECT = 5
TQ2_KERNEL_SKINNY_MMA = 6
KERNEL_NAMES = {0: "auto", 1: "gemv", 2: "skinny", 3: "tc", 4: "f32ref", 5: "tc_direct", 6: "skinny_mma"}

TQ2_F32 = 0
TQ2_F16 = 1
TQ2_BF16 = 2

# Every symbol include/tq2.h declares.
EXPORTS = (
    "tq2_soa_bytes", "tq2_status_string", "tq2_reformat_aos_to_soa", "tq2_gemv", "tq2_gemv_resident",
    "tq2_gemm",
    "tq2_gemm_f32ref", "tq2_gemm_with", "tq2_select_kernel", "tq2_set_wait_timeout_ns",
    "tq2_device_status", "tq2_version", "tq2_gemm_workspace_bytes", "tq2_gemm_ws",
    "tq2_gemm_noalloc", "tq2_quantize_f32", "tq2_gate_up_swiglu", "tq2_gate_up_swiglu_resident",
    "tq2_act16_from_f32",
    "tq2_act16_to_f32", "tq2_gemm_act16", "tq2_attention_f32",
    "tq2_rope_turns", "tq2_rope_axes", "tq2_kv_append", "tq2_attention_paged",
    "tq2_attention_paged_workspace_bytes",
    "tq2_moe_route", "tq2_moe_swiglu", "tq2_moe_swiglu_workspace_bytes", "tq2_sample",
)


class TQ2Error(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__(f"{what}: {status_string(status)}" if what else status_string(status))


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build the CUDA library first "
            "(python -m dit_tq2_g128_gb300.build, or __graft_entry__.build())")
    L = ctypes.CDLL(LIB_PATH)
    i64, vp, i32 = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int
    L.tq2_soa_bytes.restype = ctypes.c_size_t
    L.tq2_soa_bytes.argtypes = [i64, i64]
    L.tq2_status_string.restype = ctypes.c_char_p
    L.tq2_status_string.argtypes = [i32]
    L.tq2_reformat_aos_to_soa.restype = i32
    L.tq2_reformat_aos_to_soa.argtypes = [vp, vp, i64, i64, vp]
    for name in ("tq2_gemv", "tq2_gemv_resident"):
        f = getattr(L, name)
        f.restype = i32
        f.argtypes = [vp, vp, vp, vp, i64, i64, vp]
    for name in ("tq2_gemm", "tq2_gemm_f32ref"):
        f = getattr(L, name)
        f.restype = i32
        f.argtypes = [vp, vp, vp, vp, i64, i64, i64, vp]
    L.tq2_gemm_with.restype = i32
    L.tq2_gemm_with.argtypes = [i32, vp, vp, vp, vp, i64, i64, i64, vp]
    L.tq2_select_kernel.restype = i32
    L.tq2_select_kernel.argtypes = [i64, i64, i64]
    L.tq2_set_wait_timeout_ns.restype = ctypes.c_uint64
    L.tq2_set_wait_timeout_ns.argtypes = [ctypes.c_uint64]
    L.tq2_device_status.restype = i32
    L.tq2_device_status.argtypes = [vp]
    L.tq2_version.restype = i32
    L.tq2_version.argtypes = []
    L.tq2_gemm_workspace_bytes.restype = ctypes.c_size_t
    L.tq2_gemm_workspace_bytes.argtypes = [i64, i64, i64]
    L.tq2_gemm_ws.restype = i32
    L.tq2_gemm_ws.argtypes = [vp, vp, vp, vp, i64, i64, i64, vp, ctypes.c_size_t, vp]
    L.tq2_quantize_f32.restype = i32
    L.tq2_quantize_f32.argtypes = [vp, vp, i64, i64, vp]
    L.tq2_act16_from_f32.restype = i32
    L.tq2_act16_from_f32.argtypes = [vp, vp, i64, i64, vp]
    L.tq2_act16_to_f32.restype = i32
    L.tq2_act16_to_f32.argtypes = [vp, vp, i64, i64, vp]
    L.tq2_gemm_act16.restype = i32
    L.tq2_gemm_act16.argtypes = [vp, vp, vp, vp, i64, i64, i64, vp]
    L.tq2_attention_f32.restype = i32
    L.tq2_attention_f32.argtypes = [vp, vp, vp, vp, i64, i64, i64, vp]
    for name in ("tq2_gate_up_swiglu", "tq2_gate_up_swiglu_resident"):
        f = getattr(L, name)
        f.restype = i32
        f.argtypes = [vp, vp, vp, i64, i64, i64, vp]
    # tq2_heads, tq2_rope, tq2_batch and tq2_kv_cache go as packed bytes (see the functions that make them)
    ch = ctypes.c_char_p
    L.tq2_rope_turns.restype = i32
    L.tq2_rope_turns.argtypes = [vp, vp, i64]
    L.tq2_rope_axes.restype = i32
    L.tq2_rope_axes.argtypes = [ch, ch, ch, ch, ch, ch, vp, ch, i64, i64, i32, vp]
    L.tq2_kv_append.restype = i32
    L.tq2_kv_append.argtypes = [ch, ch, ch, ch, vp, ch, ch, ch, vp]
    L.tq2_attention_paged.restype = i32
    L.tq2_attention_paged.argtypes = [ch, ch, ch, ch, ctypes.c_float, i64, i32, vp, ctypes.c_size_t, vp]
    L.tq2_attention_paged_workspace_bytes.restype = ctypes.c_size_t
    L.tq2_attention_paged_workspace_bytes.argtypes = [i64, ch, ch]
    # tq2_experts and tq2_sampling go as packed bytes too
    L.tq2_moe_route.restype = i32
    L.tq2_moe_route.argtypes = [vp, i32, i64, vp, vp, i64, i64, i64, i32, i32, ctypes.c_float, vp]
    L.tq2_moe_swiglu.restype = i32
    L.tq2_moe_swiglu.argtypes = [ch, vp, vp, vp, vp, vp, i32, i64, i64, vp, ctypes.c_size_t, vp]
    L.tq2_moe_swiglu_workspace_bytes.restype = ctypes.c_size_t
    L.tq2_moe_swiglu_workspace_bytes.argtypes = [ch, i32, i64, i64]
    L.tq2_sample.restype = i32
    L.tq2_sample.argtypes = [vp, i32, i64, vp, ch, vp, vp, i64, i64, vp]
    L.tq2_gemm_noalloc.restype = i32
    L.tq2_gemm_noalloc.argtypes = [vp, vp, vp, vp, i64, i64, i64, vp]
    return L


lib = _load()


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


_torch = None
_current_raw_stream = None
_current_device = None


def _stream(stream):
    global _torch, _current_raw_stream, _current_device
    if stream is None:
        if _torch is None:
            try:
                import torch
            except ImportError:  # pragma: no cover
                return None
            _torch = torch
        if _current_device is None:
            # the raw handle without a Stream object around it (4 us of a call otherwise), and the device without its own
            # check of what is_initialized has said (1 us)
            _current_raw_stream = getattr(_torch._C, "_cuda_getCurrentRawStream", None)
            _current_device = getattr(_torch._C, "_cuda_getDevice", _torch.cuda.current_device)
        cuda = _torch.cuda
        if not cuda.is_initialized():
            return None
        if _current_raw_stream is not None:
            return _current_raw_stream(_current_device())
        return cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(status: int, what: str):
    if status != TQ2_OK:
        raise TQ2Error(status, what)


def status_string(status: int) -> str:
    return lib.tq2_status_string(int(status)).decode()


tq2_status_string = status_string


def tq2_soa_bytes(n: int, k: int) -> int:
    return int(lib.tq2_soa_bytes(n, k))


def tq2_version() -> int:
    return int(lib.tq2_version())


def tq2_select_kernel(m: int, n: int, k: int) -> int:
    return int(lib.tq2_select_kernel(m, n, k))


def tq2_set_wait_timeout_ns(ns: int) -> int:
    return int(lib.tq2_set_wait_timeout_ns(int(ns)))


def tq2_device_status(stream=None) -> int:
    """Synchronise ``stream`` and return (and clear) the device status word."""
    return int(lib.tq2_device_status(_stream(stream)))


def tq2_reformat_aos_to_soa(w_aos, w_soa, n: int, k: int, stream=None) -> None:
    _check(lib.tq2_reformat_aos_to_soa(_ptr(w_aos), _ptr(w_soa), n, k, _stream(stream)),
           "tq2_reformat_aos_to_soa")


def tq2_quantize_f32(w, w_aos, n: int, k: int, stream=None) -> None:
    _check(lib.tq2_quantize_f32(_ptr(w), _ptr(w_aos), n, k, _stream(stream)), "tq2_quantize_f32")


def tq2_act16_from_f32(x, x16, m: int, k: int, stream=None) -> None:
    _check(lib.tq2_act16_from_f32(_ptr(x), _ptr(x16), m, k, _stream(stream)), "tq2_act16_from_f32")


def tq2_act16_to_f32(x16, x, m: int, k: int, stream=None) -> None:
    _check(lib.tq2_act16_to_f32(_ptr(x16), _ptr(x), m, k, _stream(stream)), "tq2_act16_to_f32")


def tq2_gemm_act16(w_soa, x16, residual16, out16, m: int, n: int, k: int, stream=None) -> None:
    _check(lib.tq2_gemm_act16(_ptr(w_soa), _ptr(x16), _ptr(residual16), _ptr(out16), m, n, k,
                              _stream(stream)), "tq2_gemm_act16")


def tq2_attention_f32(q, k, v, out, heads: int, seq: int, dim: int, stream=None) -> None:
    _check(lib.tq2_attention_f32(_ptr(q), _ptr(k), _ptr(v), _ptr(out), heads, seq, dim, _stream(stream)),
           "tq2_attention_f32")


def tq2_gate_up_swiglu(w_soa, x, out, m: int, f: int, k: int, stream=None) -> None:
    _check(lib.tq2_gate_up_swiglu(_ptr(w_soa), _ptr(x), _ptr(out), m, f, k, _stream(stream)),
           "tq2_gate_up_swiglu")


def tq2_gate_up_swiglu_resident(w_soa, x, out, m: int, f: int, k: int, stream=None) -> None:
    _check(lib.tq2_gate_up_swiglu_resident(_ptr(w_soa), _ptr(x), _ptr(out), m, f, k, _stream(stream)),
           "tq2_gate_up_swiglu_resident")


def tq2_gemv(w_soa, x, residual, out, n: int, k: int, stream=None) -> None:
    _check(lib.tq2_gemv(_ptr(w_soa), _ptr(x), _ptr(residual), _ptr(out), n, k, _stream(stream)),
           "tq2_gemv")


def tq2_gemv_resident(w_soa, x, residual, out, n: int, k: int, stream=None) -> None:
    _check(lib.tq2_gemv_resident(_ptr(w_soa), _ptr(x), _ptr(residual), _ptr(out), n, k,
                                 _stream(stream)), "tq2_gemv_resident")


def tq2_gemm(w_soa, x, residual, out, m: int, n: int, k: int, stream=None) -> None:
    _check(lib.tq2_gemm(_ptr(w_soa), _ptr(x), _ptr(residual), _ptr(out), m, n, k,
                        _stream(stream)), "tq2_gemm")


def tq2_gemm_f32ref(w_soa, x, residual, out, m: int, n: int, k: int, stream=None) -> None:
    _check(lib.tq2_gemm_f32ref(_ptr(w_soa), _ptr(x), _ptr(residual), _ptr(out), m, n, k,
                               _stream(stream)), "tq2_gemm_f32ref")


def tq2_gemm_workspace_bytes(m: int, n: int, k: int) -> int:
    return int(lib.tq2_gemm_workspace_bytes(m, n, k))


def tq2_gemm_ws(w_soa, x, residual, out, m: int, n: int, k: int, workspace, workspace_bytes: int,
                stream=None) -> None:
    _check(lib.tq2_gemm_ws(_ptr(w_soa), _ptr(x), _ptr(residual), _ptr(out), m, n, k,
                           _ptr(workspace), int(workspace_bytes), _stream(stream)), "tq2_gemm_ws")


def tq2_gemm_noalloc(w_soa, x, residual, out, m: int, n: int, k: int, stream=None) -> None:
    """tq2_gemm without any device allocation (fixed library scratch; see include/tq2.h)."""
    _check(lib.tq2_gemm_noalloc(_ptr(w_soa), _ptr(x), _ptr(residual), _ptr(out), m, n, k,
                                _stream(stream)), "tq2_gemm_noalloc")


def tq2_gemm_with(kernel: int, w_soa, x, residual, out, m: int, n: int, k: int,
                  stream=None) -> None:
    _check(lib.tq2_gemm_with(int(kernel), _ptr(w_soa), _ptr(x), _ptr(residual), _ptr(out), m, n,
                             k, _stream(stream)), f"tq2_gemm_with({KERNEL_NAMES.get(kernel)})")


# ---------------------------------------------------------------------------
# Positions, key/value cache and its attention.  The C structs are passed as
# packed bytes: tq2_heads(...), tq2_rope(...), tq2_kv_cache(...) and tq2_batch(...)
# return them from the fields that include/tq2.h documents.


def tq2_heads(data, heads: int, token_stride: int, head_stride: int, dtype: int,
              _pack=struct.Struct("=qqqqi4x").pack) -> bytes:
    return _pack(_ptr(data) or 0, heads, token_stride, head_stride, dtype)


def tq2_rope(turns, axis, pairs: int, axes: int = 1, interleaved: int = 0,
             _pack=struct.Struct("=qqqii").pack) -> bytes:
    return _pack(_ptr(turns) or 0, _ptr(axis) or 0, pairs, axes, interleaved)


def tq2_kv_cache(k, v, pages: int, page_size: int, heads: int, dim: int, page_stride: int, slot_stride: int,
                 head_stride: int, dtype: int, _pack=struct.Struct("=qqqqqqqqqi4x").pack) -> bytes:
    return _pack(_ptr(k) or 0, _ptr(v) or 0, pages, page_size, heads, dim, page_stride, slot_stride, head_stride,
                 dtype)


def tq2_batch(q_start, kv_len, page_table, seqs: int, tokens: int, max_q: int, max_kv: int, table_stride: int,
              _pack=struct.Struct("=qqqqqqqq").pack) -> bytes:
    return _pack(_ptr(q_start) or 0, _ptr(kv_len) or 0, _ptr(page_table) or 0, seqs, tokens, max_q, max_kv,
                 table_stride)


def tq2_rope_turns(inv_freq):
    """Host: the 64-bit fractions of a turn (numpy uint64) of inv_freq (radians per position, numpy float64)."""
    import numpy as np
    f = np.ascontiguousarray(inv_freq, dtype=np.float64).reshape(-1)
    turns = np.empty(f.size, dtype=np.uint64)
    _check(lib.tq2_rope_turns(f.ctypes.data, turns.ctypes.data, f.size), "tq2_rope_turns")
    return turns


def tq2_rope_axes(q, q_out, k, k_out, v, v_out, positions, rope: bytes, tokens: int, dim: int, inverse: int = 0,
                  stream=None) -> None:
    _check(lib.tq2_rope_axes(q, q_out, k, k_out, v, v_out, _ptr(positions), rope, tokens, dim, inverse,
                             _stream(stream)), "tq2_rope_axes")


def tq2_kv_append(q, q_out, k, v, positions, rope, batch: bytes, cache: bytes, stream=None) -> None:
    _check(lib.tq2_kv_append(q, q_out, k, v, _ptr(positions), rope, batch, cache, _stream(stream)), "tq2_kv_append")


def tq2_attention_paged(q, out, cache: bytes, batch: bytes, scale: float, window: int = 0, causal: int = 1,
                        workspace=None, workspace_bytes: int = 0, stream=None) -> None:
    _check(lib.tq2_attention_paged(q, out, cache, batch, scale, window, causal, _ptr(workspace), workspace_bytes,
                                   _stream(stream)), "tq2_attention_paged")


def tq2_attention_paged_workspace_bytes(heads: int, cache: bytes, batch: bytes) -> int:
    return int(lib.tq2_attention_paged_workspace_bytes(heads, cache, batch))


# ---------------------------------------------------------------------------
# Mixtures of experts and sampling; tq2_experts(...) and tq2_sampling(...) return the C structs as packed bytes.


def tq2_experts(gate_up, down, experts: int, width: int, ffn: int, _pack=struct.Struct("=qqqqq").pack) -> bytes:
    return _pack(_ptr(gate_up) or 0, _ptr(down) or 0, experts, width, ffn)


def tq2_sampling(temperature=None, top_k=None, top_p=None, min_p=None, _pack=struct.Struct("=qqqq").pack) -> bytes:
    return _pack(_ptr(temperature) or 0, _ptr(top_k) or 0, _ptr(top_p) or 0, _ptr(min_p) or 0)


def tq2_moe_route(logits, dtype: int, row_stride: int, experts, weights, tokens: int, n_experts: int, top_k: int,
                  sigmoid: int = 0, normalize: int = 1, scale: float = 1.0, stream=None) -> None:
    _check(lib.tq2_moe_route(_ptr(logits), dtype, row_stride, _ptr(experts), _ptr(weights), tokens, n_experts, top_k,
                             sigmoid, normalize, scale, _stream(stream)), "tq2_moe_route")


def tq2_moe_swiglu(w: bytes, x, expert, weight, residual, out, dtype: int, tokens: int, top_k: int, workspace=None,
                   workspace_bytes: int = 0, stream=None) -> None:
    _check(lib.tq2_moe_swiglu(w, _ptr(x), _ptr(expert), _ptr(weight), _ptr(residual), _ptr(out), dtype, tokens, top_k,
                              _ptr(workspace), workspace_bytes, _stream(stream)), "tq2_moe_swiglu")


def tq2_moe_swiglu_workspace_bytes(w: bytes, dtype: int, tokens: int, top_k: int) -> int:
    return int(lib.tq2_moe_swiglu_workspace_bytes(w, dtype, tokens, top_k))


def tq2_sample(logits, dtype: int, row_stride: int, u, filters, tokens, prob, rows: int, vocab: int, stream=None) -> None:
    _check(lib.tq2_sample(_ptr(logits), dtype, row_stride, _ptr(u), filters, _ptr(tokens), _ptr(prob), rows, vocab,
                          _stream(stream)), "tq2_sample")


# ---------------------------------------------------------------------------
# Tensor-level conveniences (shape and dtype checks, then the calls above).  A tensor that a function makes belongs to
# the stream it runs on: to ``stream`` if given, as if made under ``torch.cuda.stream(stream)``.


def _on(stream):
    """Context whose allocations are ordered with the work of ``stream`` (None: the current one)."""
    if stream is None:
        return contextlib.nullcontext()
    import torch
    if not isinstance(stream, torch.cuda.Stream):  # (ExternalStream(0) is not the default stream)
        stream = torch.cuda.ExternalStream(_stream(stream)) if _stream(stream) else torch.cuda.default_stream()
    return torch.cuda.stream(stream)


def _check_tensor(t, name, dtype, numel):
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor")
    if str(t.dtype) != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.numel() != numel:
        raise ValueError(f"{name} has {t.numel()} elements, expected {numel}")


def upload_weight(w_aos_host, n: int, k: int, stream=None):
    """Copy AoS blocks (numpy uint8 or torch CPU tensor) to the device and
    relayout them to SoA; returns the SoA uint8 CUDA tensor (caller-owned)."""
    import numpy as np
    import torch
    nbytes = tq2_soa_bytes(n, k)
    if nbytes == 0 and n:
        raise TQ2Error(TQ2_ERR_BAD_K, "upload_weight")
    src = torch.from_numpy(np.ascontiguousarray(w_aos_host, dtype=np.uint8).reshape(-1)) \
        if not isinstance(w_aos_host, torch.Tensor) else w_aos_host.reshape(-1)
    if src.numel() != nbytes:
        raise ValueError(f"weight has {src.numel()} bytes, expected {nbytes}")
    with _on(stream):
        aos = src.to("cuda", non_blocking=False)
        soa = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    tq2_reformat_aos_to_soa(aos, soa, n, k, stream)
    return soa


def workspace(m: int, n: int, k: int, device="cuda"):
    """A device workspace for tq2_gemm_ws (torch uint8 tensor; None if not needed)."""
    import torch
    nbytes = tq2_gemm_workspace_bytes(m, n, k)
    return torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None


def matmul(w_soa, x, residual=None, *, n: int, k: int, out=None, kernel: int = TQ2_KERNEL_AUTO,
           workspace=None, stream=None):
    """out[M, N] = x[M, K] . dequant(W)^T (+ residual) on torch CUDA tensors.

    With ``workspace`` (see ``workspace()``) and kernel AUTO, runs tq2_gemm_ws."""
    import torch
    m = x.numel() // k if k else 0
    _check_tensor(w_soa, "w_soa", "torch.uint8", tq2_soa_bytes(n, k))
    _check_tensor(x, "x", "torch.float32", m * k)
    if residual is not None:
        _check_tensor(residual, "residual", "torch.float32", m * n)
    if out is None:
        with _on(stream):
            out = torch.empty((m, n), dtype=torch.float32, device=x.device)
    _check_tensor(out, "out", "torch.float32", m * n)
    if workspace is not None and kernel == TQ2_KERNEL_AUTO:
        tq2_gemm_ws(w_soa, x, residual, out, m, n, k, workspace, workspace.numel(), stream)
    else:
        tq2_gemm_with(kernel, w_soa, x, residual, out, m, n, k, stream)
    return out


# ---------------------------------------------------------------------------
# Positions, key/value cache and its attention on torch tensors.

_DTYPE = {}


def _dtype_of(t) -> int:
    if not _DTYPE:
        import torch
        _DTYPE.update({torch.float32: TQ2_F32, torch.float16: TQ2_F16, torch.bfloat16: TQ2_BF16})
    try:
        return _DTYPE[t.dtype]
    except KeyError:
        raise ValueError(f"float32, float16 or bfloat16 expected, got {t.dtype}") from None


def _heads(t, name: str, tokens: int, dim: int, _pack=struct.Struct("=qqqqi4x").pack) -> bytes:
    """The tq2_heads of a [tokens, heads, dim] CUDA tensor (any strides, the last one 1)."""
    shape, strides = t.shape, t.stride()
    if len(shape) != 3 or shape[0] != tokens or shape[2] != dim or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor [{tokens}, heads, {dim}], got {t.device} {tuple(shape)}")
    if strides[2] != 1 and dim != 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    return _pack(t.data_ptr(), shape[1], strides[0], strides[1], _DTYPE[t.dtype] if t.dtype in _DTYPE else _dtype_of(t))


def _table(t, name: str, dtype: str, ndim: int):
    if not t.is_cuda or str(t.dtype) != dtype or t.dim() != ndim or (t.numel() and t.shape[-1] > 1 and t.stride(-1) != 1):
        raise ValueError(f"{name} must be a CUDA {dtype} tensor of {ndim} dimension(s) with a contiguous last one")
    return t


def _rows_inside(t, width: int) -> bool:
    """Whether rows of ``width`` elements, the last one too, lie inside t's memory (lengths are clamped to whole rows)."""
    return (t.storage_offset() + t.shape[0] * width) * t.element_size() <= t.untyped_storage().nbytes()


class Rope:
    """Rotary positions: ``inv_freq`` (radians per position of each pair of a head, host values or a tensor), the axis
    of each pair (``axis``, default 0 for all) among ``axes`` positions per token, and whether pairs are neighbours
    (``interleaved``) or lie half the rotated width apart.  Holds the device table; see tq2_rope in include/tq2.h."""

    def __init__(self, inv_freq, axis=None, *, axes: int = 1, interleaved: bool = False, device="cuda"):
        import numpy as np
        import torch
        f = inv_freq.detach().cpu().numpy() if isinstance(inv_freq, torch.Tensor) else inv_freq
        turns = tq2_rope_turns(np.asarray(f, dtype=np.float64))
        self.pairs, self.axes, self.interleaved = int(turns.size), int(axes), bool(interleaved)
        self.turns = torch.from_numpy(turns.view(np.int64)).to(device)
        self.axis = None
        if axis is not None:
            a = torch.as_tensor(axis).detach().cpu().reshape(-1)
            if a.numel() != self.pairs or (self.pairs and not 0 <= int(a.min()) <= int(a.max()) < self.axes):
                raise ValueError(f"axis must hold {self.pairs} values from 0 to {self.axes - 1}")
            self.axis = a.to(torch.uint8).to(device)
        self._int64 = torch.int64
        self.packed = tq2_rope(self.turns, self.axis, self.pairs, self.axes, int(self.interleaved))

    def positions(self, positions, tokens: int):
        """``positions`` as checked int64 [tokens, axes] (one axis: [tokens] too), or None."""
        if positions is None:
            return None
        if (positions.dtype is not self._int64 or not positions.is_cuda or not positions.is_contiguous()
                or positions.numel() != tokens * self.axes or (self.axes > 1 and positions.shape[-1] != self.axes)):
            raise ValueError(f"positions must be a contiguous CUDA int64 tensor [{tokens}, {self.axes}]")
        return positions


class KVCache:
    """A paged cache: ``k`` and ``v`` of shape [pages, page_size, heads, dim] and the same strides (transposed views of
    [pages, heads, page_size, dim] included), float16 or bfloat16.  Holds the tensors; see tq2_kv_cache."""

    def __init__(self, k, v):
        if k.dim() != 4 or k.shape != v.shape or k.stride() != v.stride() or k.dtype != v.dtype:
            raise ValueError("k and v must be [pages, page_size, heads, dim] tensors of one type, shape and strides")
        if not (k.is_cuda and v.is_cuda) or (k.stride(3) != 1 and k.shape[3] != 1):
            raise ValueError("k and v must be CUDA tensors with a contiguous last dimension")
        self.k, self.v = k, v
        self.pages, self.page_size, self.heads, self.dim = (int(n) for n in k.shape)
        self.dtype = k.dtype
        self.packed = tq2_kv_cache(k, v, self.pages, self.page_size, self.heads, self.dim, *k.stride()[:3],
                                   _dtype_of(k))


class PagedBatch:
    """The sequences of one step: int32 device tables ``q_start`` [seqs + 1], ``kv_len`` [seqs] (the new tokens'
    keys included) and ``page_table`` [seqs, entries] (contiguous, or the first columns of a wider one), with the host's
    bounds.  Holds the tables, whose values may change between calls (a captured graph reads them anew); see tq2_batch."""

    def __init__(self, q_start, kv_len, page_table, *, tokens: int, max_q: int, max_kv: int):
        _table(q_start, "q_start", "torch.int32", 1)
        _table(kv_len, "kv_len", "torch.int32", 1)
        _table(page_table, "page_table", "torch.int32", 2)
        seqs = kv_len.numel()
        if q_start.numel() != seqs + 1 or page_table.shape[0] != seqs:
            raise ValueError(f"{seqs} sequences need q_start [{seqs + 1}] and page_table [{seqs}, entries]")
        width = page_table.stride(0) if seqs > 1 else page_table.shape[1]
        if width < page_table.shape[1] or (width > page_table.shape[1] and not _rows_inside(page_table, width)):
            raise ValueError("page_table must be contiguous, or the first columns of a wider table")
        self.q_start, self.kv_len, self.page_table = q_start, kv_len, page_table
        self.seqs, self.tokens, self.max_q, self.max_kv = int(seqs), int(tokens), int(max_q), int(max_kv)
        self.packed = tq2_batch(q_start, kv_len, page_table, self.seqs, self.tokens, self.max_q, self.max_kv, width)


def rope_axes(q, k=None, v=None, *, positions, rope: Rope, out=None, inverse: bool = False, stream=None):
    """Rotate q and k [tokens, heads, dim] by their positions and copy v, into ``out`` (a sequence of as many tensors,
    of any layout and another type if wanted; default: new contiguous ones).  Returns the outputs as a tuple.
    ``inverse`` is the gradient: the gradients of the outputs go in, those of the inputs come out.  (Autograd does not
    record the call: outputs of tensors that require a gradient have none, and the backward pass is that second call.)"""
    tokens, _, dim = q.shape
    ins = [t for t in (q, k, v) if t is not None]
    if out is None:
        import torch
        with _on(stream):
            out = [torch.empty(t.shape, dtype=t.dtype, device=t.device) for t in ins]
    if len(out) != len(ins):
        raise ValueError(f"{len(ins)} outputs expected, got {len(out)}")
    qi, qo = _heads(q, "q", tokens, dim), _heads(out[0], "q's output", tokens, dim)
    ki = ko = vi = vo = None
    if k is not None:
        ki, ko = _heads(k, "k", tokens, dim), _heads(out[1], "k's output", tokens, dim)
    if v is not None:
        vi, vo = _heads(v, "v", tokens, dim), _heads(out[-1], "v's output", tokens, dim)
    tq2_rope_axes(qi, qo, ki, ko, vi, vo, rope.positions(positions, tokens), rope.packed, tokens, dim, int(inverse), stream)
    return tuple(out)


def kv_append(k, v, cache: KVCache, batch: PagedBatch, *, rope: Rope = None, positions=None, q=None, q_out=None,
              stream=None):
    """Store a step's k (rotated by ``rope``) and v [tokens, heads, dim] in ``cache``; returns q rotated (in ``q_out``,
    default: a new tensor of the cache's type), or None without q.  ``positions`` [tokens, axes] default to each
    token's key index."""
    tokens, dim = batch.tokens, cache.dim
    qp = qo = None
    if q is not None:
        if q_out is None:
            import torch
            with _on(stream):
                q_out = torch.empty(q.shape, dtype=cache.dtype, device=q.device)
        qp, qo = _heads(q, "q", tokens, dim), _heads(q_out, "q_out", tokens, dim)
    pos = rope.positions(positions, tokens) if rope is not None else None
    tq2_kv_append(qp, qo, _heads(k, "k", tokens, dim), _heads(v, "v", tokens, dim), pos,
                  None if rope is None else rope.packed, batch.packed, cache.packed, stream)
    return q_out if q is not None else None


def attention_paged_workspace(q, cache: KVCache, batch: PagedBatch):
    """A device workspace for attention_paged of these arguments (torch uint8 tensor; None if not needed)."""
    import torch
    nbytes = tq2_attention_paged_workspace_bytes(q.shape[1], cache.packed, batch.packed)
    return torch.empty(nbytes, dtype=torch.uint8, device=q.device) if nbytes else None


def attention_paged(q, cache: KVCache, batch: PagedBatch, *, out=None, scale: float = None, window: int = 0,
                    causal: bool = True, workspace=None, stream=None):
    """Attention of the step's tokens q [tokens, heads, dim] over the paged cache, causal by default and within the
    last ``window`` keys if given; ``scale`` defaults to 1/sqrt(dim).  Returns ``out`` (default: a new tensor of q's
    type; a float32 one keeps more of the softmax's bits)."""
    if out is None:
        import torch
        with _on(stream):
            out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    tokens, dim = batch.tokens, cache.dim
    tq2_attention_paged(_heads(q, "q", tokens, dim), _heads(out, "out", tokens, dim), cache.packed, batch.packed,
                        dim ** -0.5 if scale is None else scale, window, int(causal), workspace,
                        0 if workspace is None else workspace.numel(), stream)
    return out


# ---------------------------------------------------------------------------
# Mixtures of experts and sampling on torch tensors.


def _rows(t, name: str):
    """(rows, columns, row stride, type) of a CUDA matrix with contiguous rows."""
    shape, strides = t.shape, t.stride()
    if len(shape) != 2 or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor of 2 dimensions, got {t.device} {tuple(shape)}")
    if strides[1] != 1 and shape[1] != 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    return shape[0], shape[1], strides[0], _DTYPE[t.dtype] if t.dtype in _DTYPE else _dtype_of(t)


def _given(t, name: str, dtype, shape) -> int:
    """The pointer of a contiguous CUDA tensor of this type and shape."""
    if t.dtype is not dtype or t.shape != shape or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA {dtype} tensor {tuple(shape)}, got {t.device} {t.dtype} {tuple(t.shape)}")
    return t.data_ptr()


def _made(t, name: str, dtype, shape, like, stream):
    """(tensor, pointer): t, checked, or a new tensor of this type and shape."""
    if t is not None:
        return t, _given(t, name, dtype, shape)
    if stream is None:
        t = _torch.empty(shape, dtype=dtype, device=like.device)
    else:
        with _on(stream):
            t = _torch.empty(shape, dtype=dtype, device=like.device)
    return t, t.data_ptr()


def _types():
    """torch's int32, int64 and float32 (torch is imported by whoever holds tensors)."""
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    return _torch.int32, _torch.int64, _torch.float32


def moe_route(logits, top_k: int, *, sigmoid: bool = False, normalize: bool = True, scale: float = 1.0, experts=None,
              weights=None, stream=None):
    """The ``top_k`` experts of each token by the router's logits [tokens, experts] (float32, float16 or bfloat16; rows
    of any stride), and their weights: softmax or ``sigmoid`` scores, over their sum if ``normalize``, times ``scale``.
    Returns int32 and float32 tensors [tokens, top_k] (``experts`` and ``weights`` if given); see tq2_moe_route."""
    tokens, n, stride, dtype = _rows(logits, "logits")
    i32, _, f32 = _types()
    shape = (tokens, top_k)
    experts, ep = _made(experts, "experts", i32, shape, logits, stream)
    weights, wp = _made(weights, "weights", f32, shape, logits, stream)
    status = lib.tq2_moe_route(logits.data_ptr(), dtype, stride, ep, wp, tokens, n, top_k, sigmoid, normalize, scale,
                               _stream(stream))
    if status:
        raise TQ2Error(status, "tq2_moe_route")
    return experts, weights


class Experts:
    """The ternary weights of a mixture's experts in the device layout (upload_weight): ``gate_up`` of experts * 2 * ffn
    rows (each expert's gate projection, then its up projection) of ``width`` columns, ``down`` of experts * width rows
    of ``ffn`` columns.  Holds the tensors; see tq2_experts in include/tq2.h."""

    def __init__(self, gate_up, down, *, experts: int, width: int, ffn: int):
        self.experts, self.width, self.ffn = int(experts), int(width), int(ffn)
        for t, name, rows, cols in ((gate_up, "gate_up", self.experts * 2 * self.ffn, self.width),
                                    (down, "down", self.experts * self.width, self.ffn)):
            nbytes = tq2_soa_bytes(rows, cols)
            if nbytes == 0:
                raise TQ2Error(TQ2_ERR_BAD_K, "Experts")
            _check_tensor(t, name, "torch.uint8", nbytes)
        self.gate_up, self.down = gate_up, down
        self.packed = tq2_experts(gate_up, down, self.experts, self.width, self.ffn)


def moe_swiglu_workspace(experts: Experts, tokens: int, top_k: int, dtype):
    """A device workspace for moe_swiglu of up to ``tokens`` tokens of this torch type (None if not needed)."""
    import torch
    nbytes = tq2_moe_swiglu_workspace_bytes(experts.packed, _dtype_of(torch.empty(0, dtype=dtype)), tokens, top_k)
    return torch.empty(nbytes, dtype=torch.uint8, device=experts.down.device) if nbytes else None


def moe_swiglu(layer: Experts, x, expert, weight, *, residual=None, out=None, workspace=None, stream=None):
    """A mixture-of-experts layer on tokens x [tokens, width] (float32, float16 or bfloat16), routed to ``expert`` (int32
    [tokens, top_k]; -1: none) with ``weight`` (float32): the weighted sum of their SwiGLU products (+ residual).
    Returns ``out`` (default: a new tensor; it may be the residual)."""
    tokens, width, stride, dtype = _rows(x, "x")
    if width != layer.width or (stride != width and tokens > 1):
        raise ValueError(f"x must be a contiguous tensor [tokens, {layer.width}], got {tuple(x.shape)}")
    routed = expert.shape
    if len(routed) != 2 or routed[0] != tokens:
        raise ValueError(f"expert must be [{tokens}, top_k], got {tuple(routed)}")
    i32, _, f32 = _types()
    out, op = _made(out, "out", x.dtype, x.shape, x, stream)
    status = lib.tq2_moe_swiglu(layer.packed, x.data_ptr(), _given(expert, "expert", i32, routed),
                                _given(weight, "weight", f32, routed),
                                None if residual is None else _given(residual, "residual", x.dtype, x.shape), op, dtype,
                                tokens, routed[1], None if workspace is None else workspace.data_ptr(),
                                0 if workspace is None else workspace.numel(), _stream(stream))
    if status:
        raise TQ2Error(status, "tq2_moe_swiglu")
    return out


def sample(logits, u, *, temperature=None, top_k=None, top_p=None, min_p=None, out=None, prob=None, stream=None):
    """One token of each row of logits [rows, vocab] (float32, float16 or bfloat16; rows of any stride) by random numbers
    ``u`` (float32 [rows], in [0, 1)).  The filters are CUDA tensors [rows] (float32, top_k int32), None where off.
    Returns int64 tokens and the float32 probabilities with which they were drawn, [rows] each (``out`` and ``prob`` if
    given); see tq2_sample."""
    rows, vocab, stride, dtype = _rows(logits, "logits")
    i32, i64, f32 = _types()
    shape = (rows,)
    out, op = _made(out, "out", i64, shape, logits, stream)
    prob, pp = _made(prob, "prob", f32, shape, logits, stream)
    filters = tq2_sampling(None if temperature is None else _given(temperature, "temperature", f32, shape),
                           None if top_k is None else _given(top_k, "top_k", i32, shape),
                           None if top_p is None else _given(top_p, "top_p", f32, shape),
                           None if min_p is None else _given(min_p, "min_p", f32, shape))
    status = lib.tq2_sample(logits.data_ptr(), dtype, stride, _given(u, "u", f32, shape), filters, op, pp, rows, vocab,
                            _stream(stream))
    if status:
        raise TQ2Error(status, "tq2_sample")
    return out, prob
