"""Python binding of the GB300 low-bit product library (liblb.so, C ABI in include/lb.h).

The functions here carry the C names and only marshal arguments: torch tensors (or raw integer
device addresses) become pointers, the stream defaults to torch's current CUDA stream, and a
non-zero status raises :class:`LBError`.  Every step of the computation runs in the library's
CUDA kernels; there is no CPU or PyTorch fallback.  If the library is missing it is built with
nvcc on first use; if that fails, or the device is not sm_103, the call raises.
"""
from __future__ import annotations

import ctypes
import os
import threading

from . import build as _build

__all__ = [
    "LBError", "load", "library_path", "status_string", "scale_stride", "lb_device_status",
    "lb_quantize_q8_0", "lb_quantize_i8_absmax", "lb_repack_q1_0", "lb_repack_q2_0_g64",
    "lb_gemv_q1_0", "lb_gemv_q2_0_g64", "lb_gemv_trit_planes", "lb_gemv_bf16",
    "lb_gemv_q1_0_grouped", "lb_gemv_q2_0_g64_grouped", "lb_gemv_trit_planes_grouped",
    "lb_gemm_workspace_bytes", "lb_gemm_q1_0", "lb_gemm_q2_0_g64", "lb_gemm_q1_0_grouped",
    "lb_gemm_q2_0_g64_grouped", "lb_gemm_q2_0_g64_noalloc", "lb_gemm_trit_workspace_bytes",
    "lb_gemm_trit_planes", "lb_gemm_trit_planes_grouped", "lb_quantize_i8_absmax_tiles",
    "lb_gemm_trit_planes_grouped_tiles", "lb_dequantize_q1_0",
    "lb_dequantize_q2_0_g64", "lb_dequantize_trit_planes", "OUT_F32", "OUT_BF16",
    "lb_pack_base3", "lb_gemv_base3", "base3_row_bytes", "lb_test_inject_wait_timeout",
    "lb_kv_plan", "lb_kv4_append", "lb_dequantize_kv4", "lb_attn_kv4_workspace_bytes",
    "lb_attn_kv4", "lb_logits_adjust", "kv4_cache_bytes",
    "lb_gemv_q4", "lb_gemm_q4_workspace_bytes", "lb_gemm_q4", "lb_route_workspace_bytes", "lb_route",
    "lb_experts_q4_workspace_bytes", "lb_experts_q4", "ROUTE_SOFTMAX", "ROUTE_SIGMOID",
]

LB_STATUS = {0: "LB_OK", -1: "LB_ERR_NULL", -2: "LB_ERR_ALIGN", -3: "LB_ERR_SHAPE",
             -4: "LB_ERR_BATCH", -5: "LB_ERR_ARCH", -6: "LB_ERR_LAUNCH", -7: "LB_ERR_DEVICE"}


class LBError(RuntimeError):
    def __init__(self, fn: str, status: int, cuda_error: str = ""):
        self.status = status
        self.cuda_error = cuda_error
        extra = f", {cuda_error}" if cuda_error else ""
        super().__init__(
            f"{fn} returned {status} ({LB_STATUS.get(status, 'LB_ERR_UNKNOWN')}{extra})")


_lib = None
_lock = threading.Lock()
P = ctypes.c_void_p
I64 = ctypes.c_int64
I32 = ctypes.c_int
F32 = ctypes.c_float

MAX_GROUP = 64


class lb_q_matrix(ctypes.Structure):
    _fields_ = [("bits", P), ("scales", P), ("y", P), ("isum_opt", P), ("N", I64)]


class lb_trit_matrix(ctypes.Structure):
    _fields_ = [("planes", P), ("w_scale", F32), ("y", P), ("acc_opt", P), ("N", I64)]


class lb_gemm_matrix(ctypes.Structure):
    _fields_ = [("bits", P), ("scales", P), ("y", P), ("N", I64)]


class lb_logit_rules(ctypes.Structure):
    _fields_ = [("prompt_ids", P), ("prompt_start", P), ("output_ids", P), ("output_start", P),
                ("repetition", P), ("presence", P), ("frequency", P), ("bias_ids", P),
                ("bias_values", P), ("bias_start", P), ("mask", P), ("mask_stride", I64),
                ("mask_rows", I64), ("mask_row_opt", P)]


class lb_route_rules(ctypes.Structure):
    _fields_ = [("scoring", I32), ("groups", I32), ("keep_groups", I32), ("group_best", I32),
                ("renormalize", I32), ("scale", F32), ("bias_opt", P), ("live_opt", P)]


GEMM_MAX_GROUP = 8


SIGNATURES = {
    "lb_status_string": (ctypes.c_char_p, [I32]),
    "lb_version": (I32, []),
    "lb_last_cuda_error": (I32, []),
    "lb_cuda_error_name": (ctypes.c_char_p, [I32]),
    "lb_quantize_q8_0": (I32, [P, P, P, I64, I64, P]),
    "lb_quantize_i8_absmax": (I32, [P, P, P, I64, I64, P]),
    "lb_repack_q1_0": (I32, [P, I64, I64, P, P, P]),
    "lb_repack_q2_0_g64": (I32, [P, I64, I64, P, P, P]),
    "lb_gemv_q1_0": (I32, [P, P, P, P, P, P, I64, I64, I32, P]),
    "lb_gemv_q2_0_g64": (I32, [P, P, P, P, P, P, I64, I64, I32, P]),
    "lb_gemv_trit_planes": (I32, [P, F32, P, P, P, P, I64, I64, I32, P]),
    "lb_gemv_bf16": (I32, [P, P, P, I64, I64, I32, P]),
    "lb_device_status": (I32, [P]),
    "lb_test_inject_wait_timeout": (I32, [I32]),
    "lb_gemv_q1_0_grouped": (I32, [ctypes.POINTER(lb_q_matrix), I32, P, P, I64, I32, P]),
    "lb_gemv_q2_0_g64_grouped": (I32, [ctypes.POINTER(lb_q_matrix), I32, P, P, I64, I32, P]),
    "lb_gemv_trit_planes_grouped": (I32, [ctypes.POINTER(lb_trit_matrix), I32, P, P, I64, I32,
                                          P]),
    "lb_gemm_workspace_bytes": (ctypes.c_size_t, [I64, I64]),
    "lb_gemm_q1_0": (I32, [P, P, P, P, P, I64, I64, I64, P, ctypes.c_size_t, P]),
    "lb_gemm_q2_0_g64": (I32, [P, P, P, P, P, I64, I64, I64, P, ctypes.c_size_t, P]),
    "lb_gemm_q2_0_g64_noalloc": (I32, [P, P, P, P, P, I64, I64, I64, P]),
    "lb_gemm_q1_0_grouped": (I32, [ctypes.POINTER(lb_gemm_matrix), I32, P, P, I64, I64, P,
                                   ctypes.c_size_t, P]),
    "lb_gemm_q2_0_g64_grouped": (I32, [ctypes.POINTER(lb_gemm_matrix), I32, P, P, I64, I64, P,
                                       ctypes.c_size_t, P]),
    "lb_gemm_trit_workspace_bytes": (ctypes.c_size_t, [I64, I64]),
    "lb_gemm_trit_planes": (I32, [P, F32, P, P, P, P, I64, I64, I64, P, ctypes.c_size_t, P]),
    "lb_gemm_trit_planes_grouped": (I32, [ctypes.POINTER(lb_trit_matrix), I32, P, P, I64, I64, P,
                                          ctypes.c_size_t, P]),
    "lb_quantize_i8_absmax_tiles": (I32, [P, P, P, I64, I64, P, ctypes.c_size_t, P]),
    "lb_gemm_trit_planes_grouped_tiles": (I32, [ctypes.POINTER(lb_trit_matrix), I32, P, I64, I64,
                                                P, ctypes.c_size_t, P]),
    "lb_dequantize_q1_0": (I32, [P, P, I64, I64, I32, P, P]),
    "lb_dequantize_q2_0_g64": (I32, [P, P, I64, I64, I32, P, P]),
    "lb_dequantize_trit_planes": (I32, [P, F32, I64, I64, I32, P, P]),
    "lb_pack_base3": (I32, [P, I64, I64, P, P]),
    "lb_gemv_base3": (I32, [P, F32, P, P, P, P, I64, I64, I32, P]),
    "lb_kv_plan": (I32, [P, P, I64, P, I64, P, I32, P, I64, I64, P, P, P, P, P, P]),
    "lb_kv4_append": (I32, [P, P, I32, I64, I64, P, I64, P, I64, I32, I32, I32, P]),
    "lb_dequantize_kv4": (I32, [P, I64, I32, I32, I32, P, I64, I32, P, P, P]),
    "lb_attn_kv4_workspace_bytes": (ctypes.c_size_t, [I32, I32, I32, I64]),
    "lb_attn_kv4": (I32, [P, I32, I64, P, I64, I32, I32, I32, I32, P, I64, P, P, I64, I64, I64,
                          F32, I32, I64, P, I64, P, P, ctypes.c_size_t, P]),
    "lb_logits_adjust": (I32, [P, I32, I64, P, I64, I64, I64, ctypes.POINTER(lb_logit_rules), P]),
    "lb_gemv_q4": (I32, [P, P, P, I32, P, I32, I64, P, I64, I64, I64, I32, P]),
    "lb_gemm_q4_workspace_bytes": (ctypes.c_size_t, [I64, I64, I64, I32]),
    "lb_gemm_q4": (I32, [P, P, P, I32, P, I32, I64, P, I64, I64, I64, I64, P, ctypes.c_size_t, P]),
    "lb_route_workspace_bytes": (ctypes.c_size_t, [I64, I32]),
    "lb_route": (I32, [P, I32, I64, I64, I32, I32, ctypes.POINTER(lb_route_rules), P, P, P, P, P,
                       ctypes.c_size_t, P]),
    "lb_experts_q4_workspace_bytes": (ctypes.c_size_t, [I64, I32, I32, I64, I64, I32]),
    "lb_experts_q4": (I32, [P, I32, I64, I64, I32, I32, I64, I64, I32, P, P, P, P, P, P, P, P, P, P,
                            P, I64, P, ctypes.c_size_t, P]),
}

OUT_F32 = 0
OUT_BF16 = 1

ROUTE_SOFTMAX = 0
ROUTE_SIGMOID = 1

NOALLOC_SCRATCH_BYTES = 8 << 20


def library_path() -> str:
    return _build.LIB


def load(build_if_missing: bool = True):
    """Load liblb.so (building it with nvcc if it is missing or stale)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            path = _build.LIB
            if build_if_missing and not _build.up_to_date():
                path = _build.build()
            if not os.path.exists(path):
                raise RuntimeError(f"GB300 library not built: {path} is missing")
            lib = ctypes.CDLL(path)
            for name, (res, args) in SIGNATURES.items():
                fn = getattr(lib, name)
                fn.restype = res
                fn.argtypes = args
            _lib = lib
    return _lib


def scale_stride(K: int, qk: int) -> int:
    """Row stride (entries) of a repacked scale plane: K/QK rounded up to a multiple of 8."""
    return (K // qk + 7) // 8 * 8


def status_string(status: int) -> str:
    return load().lb_status_string(int(status)).decode()


def _ptr(t):
    if t is None:
        return None
    try:
        if t.is_cuda and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        if isinstance(t, int):
            return t
        raise TypeError(f"cannot pass {type(t)} as a device pointer") from None
    raise ValueError("lb_* entry points take contiguous tensors" if t.is_cuda else
                     "lb_* entry points take device tensors")


def _rows(t):
    """Pointer of a tensor whose first dimension may be strided (a slice of a wider buffer); what
    follows it lies together."""
    if not hasattr(t, "data_ptr"):
        return _ptr(t)
    if not t.is_cuda:
        raise ValueError("lb_* entry points take device tensors")
    if t.is_contiguous():
        return t.data_ptr()
    dense = 1
    for n, s in zip(t.shape[:0:-1], t.stride()[:0:-1]):
        if s != dense and n != 1:
            raise ValueError("only the first dimension may be strided")
        dense *= n
    return t.data_ptr()


_current_stream = None


def _find_current_stream():
    """A function that returns the address of torch's current stream (the short way to it where this
    torch has it: a call of these entry points costs a few microseconds, a Stream object three)."""
    import torch
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    device = getattr(torch._C, "_cuda_getDevice", None)
    if raw is None or device is None:
        return lambda: torch.cuda.current_stream().cuda_stream
    torch.cuda.current_stream()  # initializes CUDA
    return lambda: raw(device())


def _stream(stream):
    if stream is None:
        global _current_stream
        if _current_stream is None:
            _current_stream = _find_current_stream()
        return _current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(fn: str, status: int):
    if status != 0:
        cuda = ""
        if status == -6:  # LB_ERR_LAUNCH
            code = load().lb_last_cuda_error()
            if code:
                cuda = load().lb_cuda_error_name(code).decode()
        raise LBError(fn, status, cuda)


def lb_last_cuda_error() -> int:
    """cudaError_t of the library's last failed CUDA call on this thread (then reset), or 0."""
    return int(load().lb_last_cuda_error())


def lb_cuda_error_name(code: int) -> str:
    return load().lb_cuda_error_name(int(code)).decode()


def lb_quantize_q8_0(x, q, d, B: int, K: int, stream=None):
    _check("lb_quantize_q8_0", load().lb_quantize_q8_0(_ptr(x), _ptr(q), _ptr(d), B, K,
                                                       _stream(stream)))


def lb_quantize_i8_absmax(x, q, x_scale, B: int, K: int, stream=None):
    _check("lb_quantize_i8_absmax", load().lb_quantize_i8_absmax(
        _ptr(x), _ptr(q), _ptr(x_scale), B, K, _stream(stream)))


def lb_repack_q1_0(blocks18, N: int, K: int, bits, scales, stream=None):
    _check("lb_repack_q1_0", load().lb_repack_q1_0(_ptr(blocks18), N, K, _ptr(bits),
                                                   _ptr(scales), _stream(stream)))


def lb_repack_q2_0_g64(blocks18, N: int, K: int, codes, scales, stream=None):
    _check("lb_repack_q2_0_g64", load().lb_repack_q2_0_g64(_ptr(blocks18), N, K, _ptr(codes),
                                                           _ptr(scales), _stream(stream)))


def lb_gemv_q1_0(bits, scales, q, d, y, isum, N: int, K: int, B: int, stream=None):
    _check("lb_gemv_q1_0", load().lb_gemv_q1_0(_ptr(bits), _ptr(scales), _ptr(q), _ptr(d),
                                               _ptr(y), _ptr(isum), N, K, B, _stream(stream)))


def lb_gemv_q2_0_g64(codes, scales, q, d, y, isum, N: int, K: int, B: int, stream=None):
    _check("lb_gemv_q2_0_g64", load().lb_gemv_q2_0_g64(
        _ptr(codes), _ptr(scales), _ptr(q), _ptr(d), _ptr(y), _ptr(isum), N, K, B,
        _stream(stream)))


def lb_gemv_trit_planes(planes, w_scale: float, q, x_scale, y, acc, N: int, K: int, B: int,
                        stream=None):
    _check("lb_gemv_trit_planes", load().lb_gemv_trit_planes(
        _ptr(planes), float(w_scale), _ptr(q), _ptr(x_scale), _ptr(y), _ptr(acc), N, K, B,
        _stream(stream)))


def lb_gemv_bf16(w, x, y, N: int, K: int, B: int, stream=None):
    _check("lb_gemv_bf16", load().lb_gemv_bf16(_ptr(w), _ptr(x), _ptr(y), N, K, B,
                                               _stream(stream)))


def lb_device_status(stream=None) -> int:
    """Synchronize the stream and return (and clear) the device error status (0 = OK)."""
    return load().lb_device_status(_stream(stream))


def lb_test_inject_wait_timeout(wait_us: int):
    """Test hook: the next streaming GEMV call or 4-bit product starves its first CTA, whose bounded
    wait then gives up after wait_us microseconds (reported by lb_device_status as LB_ERR_DEVICE)."""
    _check("lb_test_inject_wait_timeout", load().lb_test_inject_wait_timeout(int(wait_us)))


def _q_mats(mats):
    if not 1 <= len(mats) <= MAX_GROUP:
        raise ValueError(f"a group holds 1..{MAX_GROUP} matrices")
    arr = (lb_q_matrix * len(mats))()
    for i, (bits, scales, y, isum, N) in enumerate(mats):
        arr[i] = lb_q_matrix(_ptr(bits), _ptr(scales), _ptr(y), _ptr(isum), int(N))
    return arr


def lb_gemv_q1_0_grouped(mats, q, d, K: int, B: int, stream=None):
    """mats: sequence of (bits, scales, y, isum_or_None, N) sharing the activation q, d."""
    arr = _q_mats(mats)
    _check("lb_gemv_q1_0_grouped", load().lb_gemv_q1_0_grouped(
        arr, len(mats), _ptr(q), _ptr(d), K, B, _stream(stream)))


def lb_gemv_q2_0_g64_grouped(mats, q, d, K: int, B: int, stream=None):
    """mats: sequence of (codes, scales, y, isum_or_None, N) sharing the activation q, d."""
    arr = _q_mats(mats)
    _check("lb_gemv_q2_0_g64_grouped", load().lb_gemv_q2_0_g64_grouped(
        arr, len(mats), _ptr(q), _ptr(d), K, B, _stream(stream)))


def lb_gemv_trit_planes_grouped(mats, q, x_scale, K: int, B: int, stream=None):
    """mats: sequence of (planes, w_scale, y, acc_or_None, N) sharing the activation."""
    if not 1 <= len(mats) <= MAX_GROUP:
        raise ValueError(f"a group holds 1..{MAX_GROUP} matrices")
    arr = (lb_trit_matrix * len(mats))()
    for i, (planes, w_scale, y, acc, N) in enumerate(mats):
        arr[i] = lb_trit_matrix(_ptr(planes), float(w_scale), _ptr(y), _ptr(acc), int(N))
    _check("lb_gemv_trit_planes_grouped", load().lb_gemv_trit_planes_grouped(
        arr, len(mats), _ptr(q), _ptr(x_scale), K, B, _stream(stream)))


def lb_gemm_workspace_bytes(M: int, K: int) -> int:
    """Bytes of device scratch lb_gemm_* needs for M tokens of K columns."""
    return int(load().lb_gemm_workspace_bytes(int(M), int(K)))


def _gemm(name, bits, scales, q, d, y, M, N, K, workspace, workspace_bytes, stream):
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    nbytes = int(workspace_bytes)
    _check(name, getattr(load(), name)(_ptr(bits), _ptr(scales), _ptr(q), _ptr(d), _ptr(y),
                                       int(M), int(N), int(K), _ptr(workspace), nbytes,
                                       _stream(stream)))


def lb_gemm_q1_0(bits, scales, q, d, y, M: int, N: int, K: int, workspace,
                 workspace_bytes=None, stream=None):
    """workspace: a device tensor (its size is passed) or a pointer with workspace_bytes."""
    _gemm("lb_gemm_q1_0", bits, scales, q, d, y, M, N, K, workspace, workspace_bytes, stream)


def lb_gemm_q2_0_g64(codes, scales, q, d, y, M: int, N: int, K: int, workspace,
                     workspace_bytes=None, stream=None):
    _gemm("lb_gemm_q2_0_g64", codes, scales, q, d, y, M, N, K, workspace, workspace_bytes,
          stream)


def _gemm_grouped(name, mats, q, d, M, K, workspace, workspace_bytes, stream):
    if not 1 <= len(mats) <= GEMM_MAX_GROUP:
        raise ValueError(f"a GEMM group holds 1..{GEMM_MAX_GROUP} matrices")
    arr = (lb_gemm_matrix * len(mats))()
    for i, (bits, scales, y, N) in enumerate(mats):
        arr[i] = lb_gemm_matrix(_ptr(bits), _ptr(scales), _ptr(y), int(N))
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    _check(name, getattr(load(), name)(arr, len(mats), _ptr(q), _ptr(d), int(M), int(K),
                                       _ptr(workspace), int(workspace_bytes), _stream(stream)))


def lb_gemm_q1_0_grouped(mats, q, d, M: int, K: int, workspace, workspace_bytes=None,
                         stream=None):
    """mats: sequence of (bits, scales, y, N) sharing the activation q, d (one launch)."""
    _gemm_grouped("lb_gemm_q1_0_grouped", mats, q, d, M, K, workspace, workspace_bytes, stream)


def lb_gemm_q2_0_g64_grouped(mats, q, d, M: int, K: int, workspace, workspace_bytes=None,
                             stream=None):
    """mats: sequence of (codes, scales, y, N) sharing the activation q, d (one launch)."""
    _gemm_grouped("lb_gemm_q2_0_g64_grouped", mats, q, d, M, K, workspace, workspace_bytes,
                  stream)


def lb_gemm_q2_0_g64_noalloc(codes, scales, q, d, y, M: int, N: int, K: int, stream=None):
    """lb_gemm_q2_0_g64 with the library's fixed scratch (no workspace argument)."""
    _check("lb_gemm_q2_0_g64_noalloc", load().lb_gemm_q2_0_g64_noalloc(
        _ptr(codes), _ptr(scales), _ptr(q), _ptr(d), _ptr(y), int(M), int(N), int(K),
        _stream(stream)))


def lb_gemm_trit_workspace_bytes(M: int, K: int) -> int:
    """Bytes of device scratch lb_gemm_trit_planes* needs for M tokens of K columns."""
    return int(load().lb_gemm_trit_workspace_bytes(int(M), int(K)))


def lb_gemm_trit_planes(planes, w_scale: float, q, x_scale, y, acc, M: int, N: int, K: int,
                        workspace, workspace_bytes=None, stream=None):
    """Planar ternary prefill GEMM; workspace: a device tensor (its size is passed) or a
    pointer with workspace_bytes."""
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    _check("lb_gemm_trit_planes", load().lb_gemm_trit_planes(
        _ptr(planes), float(w_scale), _ptr(q), _ptr(x_scale), _ptr(y), _ptr(acc), int(M),
        int(N), int(K), _ptr(workspace), int(workspace_bytes), _stream(stream)))


def lb_gemm_trit_planes_grouped(mats, q, x_scale, M: int, K: int, workspace,
                                workspace_bytes=None, stream=None):
    """mats: sequence of (planes, w_scale, y, acc_or_None, N) sharing the activation (one
    launch)."""
    if not 1 <= len(mats) <= GEMM_MAX_GROUP:
        raise ValueError(f"a GEMM group holds 1..{GEMM_MAX_GROUP} matrices")
    arr = (lb_trit_matrix * len(mats))()
    for i, (planes, w_scale, y, acc, N) in enumerate(mats):
        arr[i] = lb_trit_matrix(_ptr(planes), float(w_scale), _ptr(y), _ptr(acc), int(N))
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    _check("lb_gemm_trit_planes_grouped", load().lb_gemm_trit_planes_grouped(
        arr, len(mats), _ptr(q), _ptr(x_scale), int(M), int(K), _ptr(workspace),
        int(workspace_bytes), _stream(stream)))


def lb_quantize_i8_absmax_tiles(x, q, x_scale, M: int, K: int, workspace, workspace_bytes=None,
                                stream=None):
    """lb_quantize_i8_absmax that also writes the planar GEMM's activation operand tiles into
    workspace (for lb_gemm_trit_planes_grouped_tiles)."""
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    _check("lb_quantize_i8_absmax_tiles", load().lb_quantize_i8_absmax_tiles(
        _ptr(x), _ptr(q), _ptr(x_scale), int(M), int(K), _ptr(workspace), int(workspace_bytes),
        _stream(stream)))


def lb_gemm_trit_planes_grouped_tiles(mats, x_scale, M: int, K: int, workspace,
                                      workspace_bytes=None, stream=None):
    """lb_gemm_trit_planes_grouped from the operand tiles lb_quantize_i8_absmax_tiles wrote."""
    if not 1 <= len(mats) <= GEMM_MAX_GROUP:
        raise ValueError(f"a GEMM group holds 1..{GEMM_MAX_GROUP} matrices")
    arr = (lb_trit_matrix * len(mats))()
    for i, (planes, w_scale, y, acc, N) in enumerate(mats):
        arr[i] = lb_trit_matrix(_ptr(planes), float(w_scale), _ptr(y), _ptr(acc), int(N))
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    _check("lb_gemm_trit_planes_grouped_tiles", load().lb_gemm_trit_planes_grouped_tiles(
        arr, len(mats), _ptr(x_scale), int(M), int(K), _ptr(workspace), int(workspace_bytes),
        _stream(stream)))


def lb_dequantize_q1_0(bits, scales, N: int, K: int, out_format: int, out, stream=None):
    """Every Q1_0 weight as (float)w * d: out [N][K] fp32 (OUT_F32) or bf16 bits (OUT_BF16)."""
    _check("lb_dequantize_q1_0", load().lb_dequantize_q1_0(
        _ptr(bits), _ptr(scales), int(N), int(K), int(out_format), _ptr(out), _stream(stream)))


def lb_dequantize_q2_0_g64(codes, scales, N: int, K: int, out_format: int, out, stream=None):
    _check("lb_dequantize_q2_0_g64", load().lb_dequantize_q2_0_g64(
        _ptr(codes), _ptr(scales), int(N), int(K), int(out_format), _ptr(out), _stream(stream)))


def lb_dequantize_trit_planes(planes, w_scale: float, N: int, K: int, out_format: int, out,
                              stream=None):
    _check("lb_dequantize_trit_planes", load().lb_dequantize_trit_planes(
        _ptr(planes), float(w_scale), int(N), int(K), int(out_format), _ptr(out),
        _stream(stream)))


def base3_row_bytes(K: int) -> int:
    """Bytes per base-3 packed row (LB_BASE3_ROW_BYTES): ceil(K / 80) groups of 16."""
    return (int(K) + 79) // 80 * 16


def lb_pack_base3(planes, N: int, K: int, packed, stream=None):
    _check("lb_pack_base3", load().lb_pack_base3(_ptr(planes), int(N), int(K), _ptr(packed),
                                                 _stream(stream)))


def lb_gemv_base3(packed, w_scale: float, q, x_scale, y, acc, N: int, K: int, B: int,
                  stream=None):
    _check("lb_gemv_base3", load().lb_gemv_base3(
        _ptr(packed), float(w_scale), _ptr(q), _ptr(x_scale), _ptr(y), _ptr(acc), int(N),
        int(K), int(B), _stream(stream)))


def kv4_cache_bytes(pages: int, kv_heads: int, page_size: int, head_dim: int) -> int:
    """Bytes of a 4-bit key/value cache (LB_KV4_CACHE_BYTES)."""
    return int(pages) * int(kv_heads) * int(page_size) * (int(head_dim) + 8)


def lb_kv_plan(past, fresh, R: int, free_pages, n_free: int, free_from, page_size: int,
               block_table, table_width: int, T: int, q_start, kv_len, position, slot, counts,
               stream=None):
    """Pages and slots of a step's new tokens.  free_from: None or a one-element tensor."""
    _check("lb_kv_plan", load().lb_kv_plan(
        _ptr(past), _ptr(fresh), int(R), _ptr(free_pages), int(n_free), _ptr(free_from),
        int(page_size), _ptr(block_table), int(table_width), int(T), _ptr(q_start), _ptr(kv_len),
        _ptr(position), _ptr(slot), _ptr(counts), _stream(stream)))


def lb_kv4_append(k, v, type: int, k_stride: int, v_stride: int, slot, T: int, cache, pages: int,
                  page_size: int, kv_heads: int, head_dim: int, stream=None):
    """New keys and values [T][kv_heads][head_dim] (OUT_F32 or OUT_BF16, tokens strided) -> cache."""
    _check("lb_kv4_append", load().lb_kv4_append(
        _rows(k), _rows(v), int(type), int(k_stride), int(v_stride), _ptr(slot), int(T),
        _ptr(cache), int(pages), int(page_size), int(kv_heads), int(head_dim), _stream(stream)))


def lb_dequantize_kv4(cache, pages: int, page_size: int, kv_heads: int, head_dim: int, slot,
                      T: int, out_format: int, k, v, stream=None):
    """Cache rows of T slots -> keys and values [T][kv_heads][head_dim]."""
    _check("lb_dequantize_kv4", load().lb_dequantize_kv4(
        _ptr(cache), int(pages), int(page_size), int(kv_heads), int(head_dim), _ptr(slot), int(T),
        int(out_format), _ptr(k), _ptr(v), _stream(stream)))


def lb_attn_kv4_workspace_bytes(heads: int, kv_heads: int, head_dim: int, max_q: int) -> int:
    """Bytes of device scratch lb_attn_kv4 needs."""
    return int(load().lb_attn_kv4_workspace_bytes(int(heads), int(kv_heads), int(head_dim),
                                                  int(max_q)))


def lb_attn_kv4(q, type: int, q_stride: int, cache, pages: int, page_size: int, heads: int,
                kv_heads: int, head_dim: int, block_table, table_width: int, q_start, kv_len,
                R: int, T: int, max_q: int, scale: float, causal: bool, window: int, out,
                out_stride: int, lse, workspace, workspace_bytes=None, stream=None):
    """Attention of T new tokens over the cache; q and out [T][heads][head_dim] of one type, tokens
    strided; lse None or [T][heads] fp32; workspace a device tensor (its size is passed) or a
    pointer with workspace_bytes."""
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    _check("lb_attn_kv4", load().lb_attn_kv4(
        _rows(q), int(type), int(q_stride), _ptr(cache), int(pages), int(page_size), int(heads),
        int(kv_heads), int(head_dim), _ptr(block_table), int(table_width), _ptr(q_start),
        _ptr(kv_len), int(R), int(T), int(max_q), float(scale), int(bool(causal)), int(window),
        _rows(out), int(out_stride), _ptr(lse), _ptr(workspace), int(workspace_bytes),
        _stream(stream)))


def lb_logits_adjust(logits, type: int, stride: int, out, out_stride: int, B: int, V: int, *,
                     prompt_ids=None, prompt_start=None, output_ids=None, output_start=None,
                     repetition=None, presence=None, frequency=None, bias_ids=None,
                     bias_values=None, bias_start=None, mask=None, mask_stride: int = 0,
                     mask_rows=None, mask_row=None, stream=None):
    """Penalties, biases and grammar masks on logits [B][V] (OUT_F32 or OUT_BF16, rows strided);
    out may be logits.  What is None is left out; mask_rows defaults to mask's rows."""
    if mask is not None and mask_rows is None:
        mask_rows = mask.numel() // int(mask_stride) if mask_stride > 0 else 0
    rules = lb_logit_rules(
        _ptr(prompt_ids), _ptr(prompt_start), _ptr(output_ids), _ptr(output_start),
        _ptr(repetition), _ptr(presence), _ptr(frequency), _ptr(bias_ids), _ptr(bias_values),
        _ptr(bias_start), _ptr(mask), int(mask_stride), int(mask_rows or 0), _ptr(mask_row))
    _check("lb_logits_adjust", load().lb_logits_adjust(
        _rows(logits), int(type), int(stride), _rows(out), int(out_stride), int(B), int(V),
        ctypes.byref(rules), _stream(stream)))


def _bytes_of(workspace, workspace_bytes):
    return int(workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes)


def lb_gemv_q4(codes, scales, zeros, group: int, x, type: int, x_stride: int, y, y_stride: int, N: int,
               K: int, B: int, stream=None):
    """y [B][N] = x [B][K] times 4-bit weights with group scales, B in 1..8; x and y of one type
    (OUT_F32 or OUT_BF16), rows strided; zeros: None or the groups' zero points."""
    _check("lb_gemv_q4", load().lb_gemv_q4(
        _ptr(codes), _ptr(scales), _ptr(zeros), int(group), _rows(x), int(type), int(x_stride), _rows(y),
        int(y_stride), int(N), int(K), int(B), _stream(stream)))


def lb_gemm_q4_workspace_bytes(M: int, N: int, K: int, type: int) -> int:
    """Bytes of device scratch lb_gemm_q4 needs."""
    return int(load().lb_gemm_q4_workspace_bytes(int(M), int(N), int(K), int(type)))


def lb_gemm_q4(codes, scales, zeros, group: int, x, type: int, x_stride: int, y, y_stride: int, M: int,
               N: int, K: int, workspace, workspace_bytes=None, stream=None):
    """lb_gemv_q4 for any number of tokens; workspace: a device tensor (its size is passed) or a
    pointer with workspace_bytes."""
    _check("lb_gemm_q4", load().lb_gemm_q4(
        _ptr(codes), _ptr(scales), _ptr(zeros), int(group), _rows(x), int(type), int(x_stride), _rows(y),
        int(y_stride), int(M), int(N), int(K), _ptr(workspace), _bytes_of(workspace, workspace_bytes),
        _stream(stream)))


def lb_route_workspace_bytes(T: int, E: int) -> int:
    """Bytes of device scratch lb_route needs."""
    return int(load().lb_route_workspace_bytes(int(T), int(E)))


def lb_route(logits, type: int, stride: int, T: int, E: int, k: int, scoring: int, ids, weights,
             expert_start, order, workspace, *, bias=None, groups: int = 1, keep_groups: int = 1,
             group_best: int = 1, renormalize: bool = True, scale: float = 1.0, live=None,
             workspace_bytes=None, stream=None):
    """Experts of T tokens from logits [T][E] (OUT_F32 or OUT_BF16, rows strided), and the pairs by
    expert; scoring ROUTE_SOFTMAX or ROUTE_SIGMOID; live: None or a one-element tensor."""
    rules = lb_route_rules(int(scoring), int(groups), int(keep_groups), int(group_best),
                           int(bool(renormalize)), float(scale), _ptr(bias), _ptr(live))
    _check("lb_route", load().lb_route(
        _rows(logits), int(type), int(stride), int(T), int(E), int(k), ctypes.byref(rules), _ptr(ids),
        _ptr(weights), _ptr(expert_start), _ptr(order), _ptr(workspace),
        _bytes_of(workspace, workspace_bytes), _stream(stream)))


def lb_experts_q4_workspace_bytes(T: int, E: int, k: int, hidden: int, ffn: int, type: int) -> int:
    """Bytes of device scratch lb_experts_q4 needs."""
    return int(load().lb_experts_q4_workspace_bytes(int(T), int(E), int(k), int(hidden), int(ffn),
                                                    int(type)))


def lb_experts_q4(x, type: int, x_stride: int, T: int, E: int, k: int, hidden: int, ffn: int, group: int,
                  up, down, ids, weights, expert_start, order, y, y_stride: int, workspace,
                  workspace_bytes=None, stream=None):
    """y [T][hidden] = the weighted sum of each token's experts' gated blocks; up and down:
    (codes, scales, zeros or None) of all experts; ids, weights, expert_start and order from lb_route."""
    _check("lb_experts_q4", load().lb_experts_q4(
        _rows(x), int(type), int(x_stride), int(T), int(E), int(k), int(hidden), int(ffn), int(group),
        *(_ptr(m) for m in up), *(_ptr(m) for m in down), _ptr(ids), _ptr(weights), _ptr(expert_start),
        _ptr(order), _rows(y), int(y_stride), _ptr(workspace), _bytes_of(workspace, workspace_bytes),
        _stream(stream)))
