"""Python binding of the block-scaled quantized GEMM library (``libqgemm.so``, C ABI).

Argument marshalling only: every function here passes torch tensors' device pointers, strides
and the current CUDA stream to the C entry point of the same name and raises ``QGemmError`` on a
non-OK status.  All arithmetic runs in the library's CUDA kernels; there is no CPU fallback, and
loading fails loudly when the library has not been built (``python -m
block_scaled_quantized_tcgen05_gb300.build``).
"""
from __future__ import annotations

import ctypes
import os

from . import build as _build

__all__ = [
    "QGemmError", "QTensor", "F16", "E4M3", "INT8", "INT4", "E2M1", "BF16", "load_library", "library_path",
    "qgemm_version", "qgemm_debug_build", "qgemm_create_tensor", "qgemm_tensor_slice", "qgemm_destroy_tensor",
    "qgemm_mxfp8", "qgemm_mxfp8_scratch_bytes", "qgemm_mxfp8_host", "qgemm_mxfp4", "gemm_f16", "qgemm_w4a16", "qgemm_w4a16_f16s", "qgemm_attention", "qgemm_w8_gemv", "qgemm_dequant_debug",
    "qgemm_status_string", "qgemm_poll_device_error", "qgemm_set_wait_timeout_ns",
    "qgemm_selftest_wait_timeout", "qgemm_sm_clock_probe",
    "Rotation", "KVCache", "qgemm_create_rope", "qgemm_rope", "qgemm_create_kv_cache", "qgemm_kv_append",
    "qgemm_paged_attention_workspace", "qgemm_paged_attention", "qgemm_kv_resize", "qgemm_kv_fork",
    "qgemm_kv_compact", "qgemm_kv_copy_pages",
]

F16, E4M3, INT8, INT4, E2M1, BF16 = 0, 1, 2, 3, 4, 5
OK = 0
STATUS_NAMES = {0: "QGEMM_OK", 1: "QGEMM_ERR_INVALID_ARG", 2: "QGEMM_ERR_UNSUPPORTED_SHAPE",
                3: "QGEMM_ERR_MISALIGNED", 4: "QGEMM_ERR_UNSUPPORTED_DTYPE", 5: "QGEMM_ERR_CUDA",
                6: "QGEMM_ERR_TIMEOUT"}

_lib = None


class Epilogue(ctypes.Structure):
    """qgemm_epilogue: C = relu?(A*B [+ C_old]), one fp16 rounding."""
    _fields_ = [("accumulate", ctypes.c_int32), ("relu", ctypes.c_int32)]


class QGemmError(RuntimeError):
    def __init__(self, status: int, where: str, message: str):
        self.status = status
        self.name = STATUS_NAMES.get(status, str(status))
        super().__init__(f"{where}: {self.name}: {message}")


def debug_build_selected() -> bool:
    """QGEMM_DEBUG=1 selects the bounds-checking build libqgemm_debug.so (see build.py)."""
    return os.environ.get("QGEMM_DEBUG", "") == "1"


def library_path() -> str:
    return _build.DEBUG_LIB_PATH if debug_build_selected() else _build.LIB_PATH


def load_library():
    """Load libqgemm.so (built in-tree).  Raises if it is missing: there is no fallback."""
    global _lib
    if _lib is not None:
        return _lib
    path = library_path()
    if not os.path.exists(path):
        raise ImportError(f"{os.path.basename(path)} not built at {path}; run "
                          "`python -m block_scaled_quantized_tcgen05_gb300.build"
                          + (" --debug`" if debug_build_selected() else "`"))
    lib = ctypes.CDLL(path)
    P, I64, I32, U64 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_uint64
    S = ctypes.c_int
    D, F = ctypes.c_double, ctypes.c_float
    meta = [P, P, I64, I64, I64, P, P]       # cache, table, its stride and shape, lengths, counts
    sig = {
        "qgemm_version": (I32, []),
        "qgemm_debug_build": (I32, []),
        "qgemm_create_tensor": (S, [ctypes.POINTER(P), S, I64, I64, P, I64, P, I64, I32]),
        "qgemm_tensor_slice": (S, [P, I64, I64, I64, I64, ctypes.POINTER(P)]),
        "qgemm_destroy_tensor": (None, [P]),
        "qgemm_tensor_info": (S, [P, ctypes.POINTER(I32), ctypes.POINTER(I64),
                                  ctypes.POINTER(I64), ctypes.POINTER(P), ctypes.POINTER(I64),
                                  ctypes.POINTER(P), ctypes.POINTER(I64)]),
        "qgemm_mxfp8": (S, [P, P, P, I64, P]),
        "qgemm_mxfp8_noalloc": (S, [P, P, P, I64, P]),
        "qgemm_mxfp8_scratch_bytes": (S, [P, P, ctypes.POINTER(I64)]),
        "qgemm_mxfp8_ex": (S, [P, P, P, I64, ctypes.POINTER(Epilogue), P]),
        "qgemm_mxfp4": (S, [P, P, P, I64, P]),
        "qgemm_mxfp8_host": (S, [P, P, P, I64, P]),
        "qgemm_attention_f16": (S, [P, P, P, P] + [I64] * 12 + [ctypes.c_float, P]),
        "qgemm_w4a16_f16s": (S, [P, I64, I64, P, I64, P, I64, I64, I64, P, I64, P]),
        "qgemm_w4a16_f16s_ex": (S, [P, I64, I64, P, I64, P, I64, I64, I64, P, I64,
                                    ctypes.POINTER(Epilogue), P]),
        "qgemm_mxfp4_ex": (S, [P, P, P, I64, ctypes.POINTER(Epilogue), P]),
        "gemm_f16_ex": (S, [P, I64, P, I64, P, I64, I64, I64, I64, ctypes.POINTER(Epilogue), P]),
        "qgemm_w4a16_ex": (S, [P, I64, I64, P, P, I64, ctypes.POINTER(Epilogue), P]),
        "qgemm_w8_gemv_ex": (S, [P, I64, I64, P, P, I64, ctypes.POINTER(Epilogue), P]),
        "gemm_f16": (S, [P, I64, P, I64, P, I64, I64, I64, I64, P]),
        "qgemm_w4a16": (S, [P, I64, I64, P, P, I64, P]),
        "qgemm_w8_gemv": (S, [P, I64, I64, P, P, I64, P]),
        "qgemm_dequant_debug": (S, [P, P, P]),
        "qgemm_status_string": (ctypes.c_char_p, [S]),
        "qgemm_last_error_message": (ctypes.c_char_p, []),
        "qgemm_poll_device_error": (S, [P, ctypes.POINTER(ctypes.c_uint32)]),
        "qgemm_set_wait_timeout_ns": (None, [U64]),
        "qgemm_selftest_wait_timeout": (S, [U64, P]),
        "qgemm_sm_clock_probe": (S, [U64, P, P]),
        "qgemm_create_rope": (S, [ctypes.POINTER(P), I64, I32, D, I32, D, D, D, D, D]),
        "qgemm_destroy_rope": (None, [P]),
        "qgemm_rope": (S, [P, I64, I64, P, I64, I64, I32, I64, I64, I64, P, P, I32, P]),
        "qgemm_create_kv_cache": (S, [ctypes.POINTER(P), I32, I64, I64, I64, I64, I64, P, P,
                                      ctypes.POINTER(I64), P, P, ctypes.POINTER(I64)]),
        "qgemm_destroy_kv_cache": (None, [P]),
        "qgemm_kv_append": (S, [P, I64, P, I64, I64, P, I64, I64, I32, I64, P, P, P, I64, I64, I64,
                                P, P, I64, I64, I64, P, I64, I64, P]),
        "qgemm_paged_attention_workspace_bytes": (S, [P, I64, I64, ctypes.POINTER(I64)]),
        "qgemm_paged_attention": (S, [P, I64, I64, I32, I64, I64, P, I64, P, I64, I64, I64, P, P, P,
                                      I64, I64, P, F, I64, P, I64, P]),
        "qgemm_kv_resize": (S, meta + [P, P, I64, P]),
        "qgemm_kv_fork": (S, meta + [P, P, I64, P]),
        "qgemm_kv_compact": (S, meta + [P]),
        "qgemm_kv_copy_pages": (S, [P, P, P, I64, P]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _check(status: int, where: str):
    if status != OK:
        msg = load_library().qgemm_last_error_message().decode(errors="replace")
        raise QGemmError(status, where, msg)


def _stream(stream):
    """cudaStream_t of a torch.cuda.Stream (default: torch's current stream)."""
    if stream is None:
        import torch
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return ctypes.c_void_p(stream)
    return ctypes.c_void_p(stream.cuda_stream)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _row_stride_bytes(t) -> int:
    if t.dim() != 2:
        raise ValueError("expected a 2-D tensor")
    if t.stride(1) != 1:
        raise ValueError("inner dimension must be contiguous")
    return t.stride(0) * t.element_size()


def _ld(t) -> int:
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError("expected a 2-D row-major tensor with a contiguous inner dimension")
    return t.stride(0)


class QTensor:
    """Owning Python handle of a qgemm_tensor view; keeps the borrowed torch tensors alive."""

    def __init__(self, handle: int, dtype: int, rows: int, k: int, refs):
        self.handle = ctypes.c_void_p(handle)
        self.dtype, self.rows, self.k = dtype, rows, k
        self._refs = refs

    def close(self):
        if self.handle and self.handle.value:
            load_library().qgemm_destroy_tensor(self.handle)
            self.handle = ctypes.c_void_p(None)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def qgemm_version() -> int:
    return load_library().qgemm_version()


def qgemm_debug_build() -> bool:
    """True when the loaded library is the bounds-checking debug build."""
    return load_library().qgemm_debug_build() == 1


def qgemm_status_string(status: int) -> str:
    return load_library().qgemm_status_string(status).decode()


def qgemm_create_tensor(dtype: int, data, scales=None, rows: int | None = None,
                        k: int | None = None, block_k: int = 32) -> QTensor:
    """View of a [rows, k] quantized matrix.  ``data`` is a 2-D device tensor holding the data
    plane row-major (uint8 for E4M3 / INT8 / packed INT4 or E2M1, fp16 for F16); ``scales`` is the
    [rows, k/32] uint8 UE8M0 plane (None for F16)."""
    lib = load_library()
    rows = data.shape[0] if rows is None else rows
    if k is None:
        k = {F16: data.shape[1], E4M3: data.shape[1], INT8: data.shape[1],
             INT4: 2 * data.shape[1], E2M1: 2 * data.shape[1]}[dtype]
    out = ctypes.c_void_p()
    st = lib.qgemm_create_tensor(ctypes.byref(out), dtype, rows, k, _ptr(data),
                                 _row_stride_bytes(data), _ptr(scales),
                                 _row_stride_bytes(scales) if scales is not None else 0, block_k)
    _check(st, "qgemm_create_tensor")
    return QTensor(out.value, dtype, rows, k, (data, scales))


def qgemm_tensor_slice(t: QTensor, row0: int, nrows: int, k0: int, nk: int) -> QTensor:
    lib = load_library()
    out = ctypes.c_void_p()
    _check(lib.qgemm_tensor_slice(t.handle, row0, nrows, k0, nk, ctypes.byref(out)),
           "qgemm_tensor_slice")
    return QTensor(out.value, t.dtype, nrows, nk, t._refs)


def qgemm_destroy_tensor(t: QTensor):
    t.close()


def qgemm_mxfp8(A: QTensor, B: QTensor, C, stream=None):
    _check(load_library().qgemm_mxfp8(A.handle, B.handle, _ptr(C), _ld(C), _stream(stream)),
           "qgemm_mxfp8")
    return C


def qgemm_mxfp4(A: QTensor, B: QTensor, C, stream=None):
    """C = A B^T with E2M1 operands (UE8M0 scale per 32 along K), fp32 accumulation, fp16 out."""
    _check(load_library().qgemm_mxfp4(A.handle, B.handle, _ptr(C), _ld(C), _stream(stream)),
           "qgemm_mxfp4")
    return C


def qgemm_mxfp8_host(A: QTensor, B: QTensor, C, stream=None):
    """qgemm_mxfp8 with A, B (views of host tensors, preferably pinned) and C (a host fp16 tensor)
    in host memory: uploads, computes and downloads with the three overlapped; asynchronous on
    ``stream`` (synchronise it before reading C)."""
    if C.is_cuda:
        raise ValueError("C must be a host tensor")
    _check(load_library().qgemm_mxfp8_host(A.handle, B.handle, _ptr(C), _ld(C), _stream(stream)),
           "qgemm_mxfp8_host")
    return C


def qgemm_mxfp8_scratch_bytes(A: QTensor, B: QTensor) -> int:
    """Bytes of pooled device scratch one qgemm_mxfp8 call on these views takes (0: none)."""
    n = ctypes.c_int64(0)
    _check(load_library().qgemm_mxfp8_scratch_bytes(A.handle, B.handle, ctypes.byref(n)),
           "qgemm_mxfp8_scratch_bytes")
    return n.value


def qgemm_mxfp8_noalloc(A: QTensor, B: QTensor, C, stream=None):
    """qgemm_mxfp8 with its scale scratch in the library's fixed device buffer: allocates no
    device memory (for callers that cannot allocate mid-run); shapes needing more than 8 MiB of
    repacked scales are rejected; concurrent calls on one device must not overlap on the GPU."""
    _check(load_library().qgemm_mxfp8_noalloc(A.handle, B.handle, _ptr(C), _ld(C),
                                               _stream(stream)), "qgemm_mxfp8_noalloc")
    return C


def gemm_f16(A, B, C, stream=None):
    M, K = A.shape
    N = B.shape[1]
    _check(load_library().gemm_f16(_ptr(A), _ld(A), _ptr(B), _ld(B), _ptr(C), _ld(C), M, N, K,
                                   _stream(stream)), "gemm_f16")
    return C


def qgemm_w4a16(A, W: QTensor, C, stream=None):
    _check(load_library().qgemm_w4a16(_ptr(A), _ld(A), A.shape[0], W.handle, _ptr(C), _ld(C),
                                      _stream(stream)), "qgemm_w4a16")
    return C


def qgemm_w8_gemv(X, W: QTensor, Y, stream=None):
    _check(load_library().qgemm_w8_gemv(_ptr(X), _ld(X), X.shape[0], W.handle, _ptr(Y), _ld(Y),
                                        _stream(stream)), "qgemm_w8_gemv")
    return Y


def _epi(accumulate: bool, relu: bool):
    return ctypes.byref(Epilogue(int(bool(accumulate)), int(bool(relu))))


def qgemm_mxfp8_ex(A: QTensor, B: QTensor, C, accumulate=False, relu=False, stream=None):
    """C = relu?(A B^T [+ C]) with the MXFP8 operands of qgemm_mxfp8."""
    _check(load_library().qgemm_mxfp8_ex(A.handle, B.handle, _ptr(C), _ld(C),
                                         _epi(accumulate, relu), _stream(stream)), "qgemm_mxfp8_ex")
    return C


def qgemm_mxfp4_ex(A: QTensor, B: QTensor, C, accumulate=False, relu=False, stream=None):
    """C = relu?(A B^T [+ C]) with the MXFP4 operands of qgemm_mxfp4."""
    _check(load_library().qgemm_mxfp4_ex(A.handle, B.handle, _ptr(C), _ld(C),
                                         _epi(accumulate, relu), _stream(stream)), "qgemm_mxfp4_ex")
    return C


def gemm_f16_ex(A, B, C, accumulate=False, relu=False, stream=None):
    M, K = A.shape
    N = B.shape[1]
    _check(load_library().gemm_f16_ex(_ptr(A), _ld(A), _ptr(B), _ld(B), _ptr(C), _ld(C), M, N, K,
                                      _epi(accumulate, relu), _stream(stream)), "gemm_f16_ex")
    return C


def qgemm_w4a16_ex(A, W: QTensor, C, accumulate=False, relu=False, stream=None):
    _check(load_library().qgemm_w4a16_ex(_ptr(A), _ld(A), A.shape[0], W.handle, _ptr(C), _ld(C),
                                         _epi(accumulate, relu), _stream(stream)), "qgemm_w4a16_ex")
    return C


def qgemm_attention(Q, K, V, O, scale=None, stream=None):
    """O = softmax(scale Q K^T) V per head; Q, O [BH, Lq, 128], K, V [BH, Lk, 128] fp16 device
    tensors with a contiguous last dimension; scale defaults to 1/sqrt(128)."""
    for t in (Q, K, V, O):
        if t.dim() != 3 or t.stride(2) != 1:
            raise ValueError("expected [BH, L, d] tensors with a contiguous last dimension")
    BH, Lq, d = Q.shape
    Lk = K.shape[1]
    if scale is None:
        scale = d ** -0.5
    _check(load_library().qgemm_attention_f16(
        _ptr(Q), _ptr(K), _ptr(V), _ptr(O), BH, Lq, Lk, d, Q.stride(0), Q.stride(1),
        K.stride(0), K.stride(1), V.stride(0), V.stride(1), O.stride(0), O.stride(1),
        float(scale), _stream(stream)), "qgemm_attention_f16")
    return O


def qgemm_w4a16_f16s(A, W, S, C, stream=None):
    """C = A W^T with int4 W [N, K/2] (packed uint8) and fp16 block-32 scales S [N, K/32], each
    weight dequantised to the half nearest q * s (the custom-format escape hatch)."""
    M, K = A.shape
    N = W.shape[0]
    _check(load_library().qgemm_w4a16_f16s(_ptr(A), _ld(A), M, _ptr(W), _row_stride_bytes(W),
                                           _ptr(S), _ld(S), N, K, _ptr(C), _ld(C),
                                           _stream(stream)), "qgemm_w4a16_f16s")
    return C


def qgemm_w4a16_f16s_ex(A, W, S, C, accumulate=False, relu=False, stream=None):
    M, K = A.shape
    N = W.shape[0]
    _check(load_library().qgemm_w4a16_f16s_ex(_ptr(A), _ld(A), M, _ptr(W), _row_stride_bytes(W),
                                              _ptr(S), _ld(S), N, K, _ptr(C), _ld(C),
                                              _epi(accumulate, relu), _stream(stream)),
           "qgemm_w4a16_f16s_ex")
    return C


def qgemm_w8_gemv_ex(X, W: QTensor, Y, accumulate=False, relu=False, stream=None):
    _check(load_library().qgemm_w8_gemv_ex(_ptr(X), _ld(X), X.shape[0], W.handle, _ptr(Y), _ld(Y),
                                           _epi(accumulate, relu), _stream(stream)),
           "qgemm_w8_gemv_ex")
    return Y


def qgemm_dequant_debug(t: QTensor, out, stream=None):
    _check(load_library().qgemm_dequant_debug(t.handle, _ptr(out), _stream(stream)),
           "qgemm_dequant_debug")
    return out


def qgemm_poll_device_error(stream=None) -> int:
    """Synchronise and return (and clear) the device error word; 0 when no wait gave up."""
    code = ctypes.c_uint32(0)
    st = load_library().qgemm_poll_device_error(_stream(stream), ctypes.byref(code))
    if st not in (OK, 6):
        _check(st, "qgemm_poll_device_error")
    return code.value


def qgemm_set_wait_timeout_ns(ns: int):
    load_library().qgemm_set_wait_timeout_ns(int(ns))


def qgemm_selftest_wait_timeout(timeout_ns: int, stream=None):
    _check(load_library().qgemm_selftest_wait_timeout(int(timeout_ns), _stream(stream)),
           "qgemm_selftest_wait_timeout")


def qgemm_sm_clock_probe(window_ns: int, out, stream=None):
    """Write (SM cycles, global-timer ns) over `window_ns` into the two int64 elements of the
    device tensor `out` (from the GPU, on `stream`)."""
    _check(load_library().qgemm_sm_clock_probe(int(window_ns), _ptr(out), _stream(stream)),
           "qgemm_sm_clock_probe")


# ------------------------------------------------------------------------------ decode serving
class Rotation:
    """Owning handle of rotary frequencies (qgemm_create_rope)."""

    def __init__(self, handle: int, rot_dim: int):
        self.handle = ctypes.c_void_p(handle)
        self.rot_dim = rot_dim

    def close(self):
        if self.handle and self.handle.value:
            load_library().qgemm_destroy_rope(self.handle)
            self.handle = ctypes.c_void_p(None)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class KVCache:
    """Owning handle of a paged key-value cache view; keeps the borrowed torch tensors alive."""

    def __init__(self, handle: int, dtype: int, shape, refs):
        self.handle = ctypes.c_void_p(handle)
        self.dtype = dtype
        self.layers, self.pages, self.heads, self.page_size, self.d = shape
        self.scale = self.d ** -0.5
        self._refs = refs

    def close(self):
        if self.handle and self.handle.value:
            load_library().qgemm_destroy_kv_cache(self.handle)
            self.handle = ctypes.c_void_p(None)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


_ROPE_SCALING = {"none": 0, "linear": 1, "by_parts": 2}


# A decode step makes several of these calls per layer, each a few microseconds of GPU time: the
# marshalling reads a tensor's strides once and takes the raw current stream.
torch = None


def _load_torch():
    global torch
    import torch as th
    torch = th
    return th


def _raw_stream(stream) -> int:
    """cudaStream_t of a stream (default: torch's current one) as an integer."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream if isinstance(stream, int) else stream.cuda_stream


def _dtype16(t) -> int:
    dt = t.dtype
    if dt is torch.float16:
        return F16
    if dt is torch.bfloat16:
        return BF16
    raise ValueError(f"expected an fp16 or bf16 tensor, got {dt}")


def _on_device(t, what: str):
    """Memory the GPU can read: device memory, or pinned host memory."""
    if not t.is_pinned():
        raise ValueError(f"{what}: expected a tensor in device memory, got one on {t.device}")


def _rows3(t, what: str):
    """(pointer, token stride, head stride) of a [tokens, heads, d] tensor."""
    if not t.is_cuda:
        _on_device(t, what)
    s = t.stride()
    if len(s) != 3 or s[2] != 1 and t.shape[2] > 1:
        raise ValueError(f"{what}: expected a [tokens, heads, d] tensor with a contiguous last dimension")
    return t.data_ptr(), s[0], s[1]


def _rope(r):
    """The handle of a rotation; a closed one is not taken for none."""
    if r.handle:
        return r.handle
    raise ValueError("the rotation is closed")


def _ints(t, what: str, n: int = 0):
    if t.dtype is not torch.int32 or t.dim() != 1 or not t.is_contiguous():
        raise ValueError(f"{what}: expected a contiguous 1-D int32 tensor")
    if t.numel() < n:
        raise ValueError(f"{what}: {t.numel()} entries, {n} needed")
    if not t.is_cuda:
        _on_device(t, what)
    return t.data_ptr()


def _table(t):
    """(pointer, row stride, rows, entries a row)."""
    s = t.stride()
    if t.dtype is not torch.int32 or len(s) != 2 or s[1] != 1 and t.shape[1] > 1:
        raise ValueError("page table: expected a 2-D int32 tensor with contiguous rows")
    if not t.is_cuda:
        _on_device(t, "page table")
    shape = t.shape
    return t.data_ptr(), s[0], shape[0], shape[1]


def qgemm_create_rope(rot_dim: int, base: float = 10000.0, interleaved: bool = False,
                      scaling: str = "none", factor: float = 1.0, original_len: float = 0.0,
                      low_turns: float = 1.0, high_turns: float = 4.0, mscale: float = 1.0) -> Rotation:
    """Rotary frequencies for the first ``rot_dim`` elements of a head; ``scaling`` is "none",
    "linear" (all divided by ``factor``) or "by_parts" (slow pairs divided, fast ones kept)."""
    _load_torch()
    if scaling not in _ROPE_SCALING:
        raise ValueError(f"scaling must be one of {sorted(_ROPE_SCALING)}")
    out = ctypes.c_void_p()
    _check(load_library().qgemm_create_rope(ctypes.byref(out), rot_dim, int(bool(interleaved)), base,
                                            _ROPE_SCALING[scaling], factor, original_len, low_turns,
                                            high_turns, mscale), "qgemm_create_rope")
    return Rotation(out.value, rot_dim)


def qgemm_rope(X, positions, rope: Rotation, out=None, inverse: bool = False, stream=None):
    """X [tokens, heads, d] (fp16 or bf16) rotated to ``positions`` (int32 [tokens]), into ``out``
    (default: in place).  ``inverse`` rotates back, which is the gradient."""
    turn = _rope(rope)
    shape = X.shape
    x = _rows3(X, "X")
    y = x
    if out is not None:
        if out.shape != shape or out.dtype is not X.dtype:
            raise ValueError("out: shape and type must be X's")
        y = _rows3(out, "out")
    T, H, d = shape
    st = (_lib or load_library()).qgemm_rope(*x, *y, _dtype16(X), T, H, d, _ints(positions, "positions", T),
                                             turn, 1 if inverse else 0, _raw_stream(stream))
    if st:
        _check(st, "qgemm_rope")
    return X if out is None else out


def qgemm_create_kv_cache(k, v, k_scales=None, v_scales=None) -> KVCache:
    """View of a paged cache: ``k`` and ``v`` are [layers, pages, heads, page_size, d] device tensors
    of any strides with contiguous rows (a permuted view for another order in memory), fp16, bf16, or
    uint8 / float8_e4m3fn codes with uint8 UE8M0 scales [..., 4 bytes] in ``k_scales``, ``v_scales``."""
    _load_torch()
    if k.dim() != 5 or k.shape != v.shape or k.stride() != v.stride() or k.dtype != v.dtype:
        raise ValueError("k and v: expected two [layers, pages, heads, page_size, d] tensors of one layout")
    if k.stride(4) != 1:
        raise ValueError("rows must be contiguous")
    if k.dtype in (torch.uint8, torch.float8_e4m3fn):
        dt = E4M3
    else:
        dt = _dtype16(k)
    item = k.element_size()
    strides = (ctypes.c_int64 * 4)(*(s * item for s in k.stride()[:4]))
    sstrides = None
    if k_scales is not None or v_scales is not None:
        if k_scales is None or v_scales is None or k_scales.shape != v_scales.shape or \
                k_scales.stride() != v_scales.stride():
            raise ValueError("k_scales and v_scales: expected two tensors of one layout")
        if k_scales.dtype != torch.uint8 or k_scales.dim() != 5 or k_scales.shape[:4] != k.shape[:4] or \
                k_scales.shape[4] < k.shape[4] // 32 or k_scales.stride(4) != 1:
            raise ValueError("scales: expected uint8 [layers, pages, heads, page_size, d / 32 or more]")
        sstrides = (ctypes.c_int64 * 4)(*k_scales.stride()[:4])
    for name, t in (("k", k), ("v", v), ("k_scales", k_scales), ("v_scales", v_scales)):
        if t is not None and not t.is_cuda:
            _on_device(t, name)
    out = ctypes.c_void_p()
    _check(load_library().qgemm_create_kv_cache(ctypes.byref(out), dt, *k.shape, _ptr(k), _ptr(v), strides,
                                                _ptr(k_scales), _ptr(v_scales), sstrides),
           "qgemm_create_kv_cache")
    return KVCache(out.value, dt, tuple(k.shape), (k, v, k_scales, v_scales))


def qgemm_kv_append(kv: KVCache, layer: int, K, V, seqs, positions, table, rope: Rotation | None = None,
                    Q=None, Q_out=None, stream=None):
    """Store new keys (rotated) and values [tokens, heads, d] at ``positions`` of sequences ``seqs``,
    and rotate the tokens' queries ``Q`` [tokens, q_heads, d] into ``Q_out`` (default: in place)."""
    turn = None if rope is None else _rope(rope)
    shape = K.shape
    T = shape[0]
    dt = K.dtype
    if shape != V.shape or tuple(shape) != (T, kv.heads, kv.d) or V.dtype is not dt:
        raise ValueError(f"K and V: expected [tokens, {kv.heads}, {kv.d}] of one type")
    q = qo = (None, 0, 0)
    hq = 0
    if Q is not None:
        qshape = Q.shape
        q = qo = _rows3(Q, "Q")
        if Q_out is None:
            Q_out = Q
        elif Q_out is not Q:
            if Q_out.shape != qshape or Q_out.dtype is not dt:
                raise ValueError("Q_out: shape and type must be Q's")
            qo = _rows3(Q_out, "Q_out")
        hq = qshape[1]
        if qshape[0] != T or qshape[2] != kv.d or Q.dtype is not dt:
            raise ValueError(f"Q: expected [{T}, q_heads, {kv.d}] of K's type")
    st = (_lib or load_library()).qgemm_kv_append(
        kv.handle, layer, *_rows3(K, "K"), *_rows3(V, "V"), _dtype16(K), T, _ints(seqs, "seqs", T),
        _ints(positions, "positions", T), *_table(table), turn,
        *q, hq, *qo, _raw_stream(stream))
    if st:
        _check(st, "qgemm_kv_append")
    return Q_out


def qgemm_paged_attention_workspace(kv: KVCache, batch: int, q_heads: int):
    """A zeroed workspace for qgemm_paged_attention calls of up to ``batch`` sequences, one after
    another on one stream."""
    n = ctypes.c_int64(0)
    _check(load_library().qgemm_paged_attention_workspace_bytes(kv.handle, batch, q_heads, ctypes.byref(n)),
           "qgemm_paged_attention_workspace_bytes")
    return torch.zeros(n.value, dtype=torch.uint8, device=kv._refs[0].device)


def qgemm_paged_attention(Q, kv: KVCache, layer: int, table, lens, O, seqs=None, lse=None, scale=None,
                          window: int = 0, workspace=None, stream=None):
    """O[b] = attention of Q[b] [q_heads, d] over the first ``lens[s]`` cached tokens of sequence s =
    ``seqs[b]`` (default b), the last ``window`` of them (0: all); ``lse`` (fp32 [batch, q_heads])
    receives the log of the softmax sums.  ``workspace`` comes from qgemm_paged_attention_workspace
    (one made for the call otherwise, on the current stream)."""
    shape = Q.shape
    q = _rows3(Q, "Q")
    B, H, d = shape
    if O.shape != shape or O.dtype is not Q.dtype or d != kv.d:
        raise ValueError(f"Q and O: expected [batch, q_heads, {kv.d}] of one type")
    if lse is not None and (lse.dtype is not torch.float32 or tuple(lse.shape) != (B, H) or not lse.is_contiguous()):
        raise ValueError("lse: expected a contiguous fp32 [batch, q_heads] tensor")
    if lse is not None and not lse.is_cuda:
        _on_device(lse, "lse")
    if workspace is None:
        s = stream if stream is not None and not isinstance(stream, int) else torch.cuda.current_stream()
        if isinstance(stream, int) and stream != s.cuda_stream:
            raise ValueError("a raw stream needs a workspace of its own")
        with torch.cuda.stream(s):
            workspace = qgemm_paged_attention_workspace(kv, B, H)
    elif not workspace.is_cuda:
        _on_device(workspace, "workspace")
    t = _table(table)
    st = (_lib or load_library()).qgemm_paged_attention(
        *q, _dtype16(Q), B, H, kv.handle, layer, *t, _ints(lens, "lens", t[2]),
        None if seqs is None else _ints(seqs, "seqs", B), *_rows3(O, "O"),
        None if lse is None else lse.data_ptr(), kv.scale if scale is None else scale, window,
        workspace.data_ptr(), workspace.numel(), _raw_stream(stream))
    if st:
        _check(st, "qgemm_paged_attention")
    return O


def _meta(kv: KVCache, table, lens, refs):
    t = _table(table)
    return (kv.handle, *t, _ints(lens, "lens", t[2]), _ints(refs, "refs", kv.pages))


def qgemm_kv_resize(kv: KVCache, table, lens, refs, seqs, new_lens=None, stream=None):
    """Give sequences ``seqs`` ``new_lens`` tokens (None: free them): ``table`` [max_seqs, max_pages],
    ``lens`` [max_seqs] and ``refs`` [pages] (int32) are updated on the device."""
    n = seqs.shape[0]
    _check((_lib or load_library()).qgemm_kv_resize(
        *_meta(kv, table, lens, refs), _ints(seqs, "seqs"),
        None if new_lens is None else _ints(new_lens, "new_lens", n), n, _raw_stream(stream)), "qgemm_kv_resize")


def qgemm_kv_fork(kv: KVCache, table, lens, refs, parents, children, stream=None):
    """Make sequences ``children`` copies of ``parents``: whole pages shared, a partly filled last
    page copied."""
    n = children.shape[0]
    _check((_lib or load_library()).qgemm_kv_fork(
        *_meta(kv, table, lens, refs), _ints(parents, "parents", n), _ints(children, "children"), n,
        _raw_stream(stream)), "qgemm_kv_fork")


def qgemm_kv_compact(kv: KVCache, table, lens, refs, stream=None):
    """Move the pages in use to the front of the cache."""
    _check((_lib or load_library()).qgemm_kv_compact(*_meta(kv, table, lens, refs), _raw_stream(stream)),
           "qgemm_kv_compact")


def qgemm_kv_copy_pages(kv: KVCache, src, dst, stream=None):
    """Copy pages ``src`` to ``dst`` (int32, on the device) in every layer."""
    n = src.shape[0]
    _check((_lib or load_library()).qgemm_kv_copy_pages(kv.handle, _ints(src, "src"), _ints(dst, "dst", n), n,
                                                        _raw_stream(stream)), "qgemm_kv_copy_pages")
