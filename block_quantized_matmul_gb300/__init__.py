"""block_quantized_matmul_gb300 -- Python binding of libqmm (include/qmm.h).

Matrix multiply over block-32 quantized weights (Q4_0, Q8_0, IQ4_NL; also MXFP4, Q4_1 and the
Q4_K super-blocks) stored in the 32-row tiled layout of "Hexagon backend developer details" ("Tiled
Weight Formats") or in flat GGML rows, with activations dynamically quantized to Q8_0 blocks, on
one GB300 (sm_103a).

This module only marshals arguments: every function takes torch CUDA tensors (PyTorch provides the
device memory and the stream; the fused decode call also takes pinned host tensors for x and y),
passes raw addresses and sizes through ctypes, and raises QmmError on any status other than QMM_OK.
All computation runs in the CUDA kernels of libqmm.so; there is no CPU fallback, and the first call
fails loudly if the library is missing.

A decode step over a weight w (fp32 [N, K] on the GPU):

    flat = torch.empty(flat_size("q4_0", K, N), dtype=torch.uint8, device="cuda")
    tiled = torch.empty(tiled_size("q4_0", K, N), dtype=torch.uint8, device="cuda")
    qmm_quantize_weight("q4_0", w, N, K, K, flat)        # load time
    qmm_repack("q4_0", flat, K, N, tiled)               # load time
    qmm_matmul_f32("q4_0", tiled, K, N, x, K, M, y, N)   # y[M, N] = Q8_0(x[M, K]) @ W^T

Prefill shapes: qmm_quantize_act, then qmm_matmul_ws with a workspace of matmul_workspace_size(M, K)
bytes (or qmm_matmul, which needs none).
"""
from __future__ import annotations

import ctypes
import os

__all__ = [
    "Q4_0", "Q8_0", "IQ4_NL", "MXFP4", "Q4_1", "Q4_K", "TYPES", "QmmError", "lib", "library_path",
    "block_size", "tile_size", "tiled_size", "flat_size", "iq4nl_table", "decode_max_m",
    "qmm_quantize_weight", "qmm_repack", "qmm_unpack", "qmm_quantize_act", "qmm_matmul",
    "qmm_matmul_path", "qmm_matmul_f32", "qmm_matmul_flat", "qmm_device_status", "PATH_AUTO", "PATH_MATVEC", "PATH_GEMM",
    "matmul_workspace_size", "qmm_matmul_ws", "qmm_matmul_noalloc", "matmul_noalloc_max_workspace",
    "qmm_selftest_timeout",
    "F32", "F16", "BF16", "DTYPES", "mx4_codes_size", "mx4_scales_size", "mx4_linear_workspace_size", "qmm_mx4_quantize",
    "qmm_mx4_dequantize", "qmm_mx4_matmul", "qmm_mx4_linear", "cache_page_size", "cache_attend_workspace_size",
    "qmm_cache_write", "qmm_cache_read", "qmm_cache_attend",
]

Q4_0, Q8_0, IQ4_NL, MXFP4, Q4_1, Q4_K = 0, 1, 2, 3, 4, 5
TYPES = {"q4_0": Q4_0, "q8_0": Q8_0, "iq4_nl": IQ4_NL, "mxfp4": MXFP4, "q4_1": Q4_1, "q4_k": Q4_K}
PATH_AUTO, PATH_MATVEC, PATH_GEMM = 0, 1, 2
F32, F16, BF16 = 0, 1, 2
DTYPES = {"f32": F32, "f16": F16, "bf16": BF16}
_STATUS = {0: "QMM_OK", 1: "QMM_ERR_INVALID_ARG", 2: "QMM_ERR_UNSUPPORTED", 3: "QMM_ERR_MISALIGNED",
           4: "QMM_ERR_CUDA", 5: "QMM_ERR_TIMEOUT", 6: "QMM_ERR_RANGE", 7: "QMM_ERR_BOUNDS"}

_HERE = os.path.dirname(os.path.abspath(__file__))
# QMM_DEBUG=1 in the environment selects the build with device bounds checks (libqmm_debug.so)
library_path = os.path.join(_HERE, "libqmm_debug.so" if os.environ.get("QMM_DEBUG") == "1" else "libqmm.so")
_lib = None


class QmmError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} failed: {_STATUS.get(status, status)}")


def lib():
    """Load libqmm.so (built by build.py / __graft_entry__.build()); raises if it is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(library_path):
            raise ImportError(f"libqmm.so not built at {library_path}; run `python -m block_quantized_matmul_gb300.build`")
        L = ctypes.CDLL(library_path)
        i64, i32, vp, sz = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t
        L.qmm_status_str.argtypes = [i32]
        L.qmm_status_str.restype = ctypes.c_char_p
        for fn in ("qmm_block_size", "qmm_tile_size"):
            getattr(L, fn).argtypes = [i32]
            getattr(L, fn).restype = sz
        for fn in ("qmm_tiled_size", "qmm_flat_size"):
            getattr(L, fn).argtypes = [i32, i64, i64]
            getattr(L, fn).restype = sz
        L.qmm_iq4nl_table.argtypes = [vp]
        L.qmm_iq4nl_table.restype = None
        L.qmm_decode_max_m.argtypes = []
        L.qmm_decode_max_m.restype = i64
        L.qmm_quantize_weight.argtypes = [i32, vp, i64, i64, i64, vp, vp]
        L.qmm_repack.argtypes = [i32, vp, i64, i64, vp, vp]
        L.qmm_unpack.argtypes = [i32, vp, i64, i64, vp, vp]
        L.qmm_quantize_act.argtypes = [vp, i64, i64, i64, vp, vp, vp]
        L.qmm_matmul.argtypes = [i32, vp, i64, i64, vp, vp, i64, vp, i64, vp]
        L.qmm_matmul_f32.argtypes = [i32, vp, i64, i64, vp, i64, i64, vp, i64, vp]
        L.qmm_matmul_path.argtypes = [i32, vp, i64, i64, vp, vp, i64, vp, i64, i32, vp]
        L.qmm_matmul_flat.argtypes = [i32, vp, i64, i64, vp, vp, i64, vp, i64, vp]
        L.qmm_device_status.argtypes = [vp]
        L.qmm_selftest_timeout.argtypes = [i32, ctypes.c_uint64, vp, vp]
        L.qmm_matmul_workspace_size.argtypes = [i64, i64]
        L.qmm_matmul_workspace_size.restype = sz
        L.qmm_matmul_ws.argtypes = [i32, vp, i64, i64, vp, vp, i64, vp, i64, vp, sz, vp]
        L.qmm_matmul_noalloc.argtypes = [i32, vp, i64, i64, vp, vp, i64, vp, i64, vp]
        L.qmm_matmul_noalloc_max_workspace.argtypes = []
        L.qmm_matmul_noalloc_max_workspace.restype = sz
        L.qmm_matmul_f32_workspace_size.argtypes = [i64, i64]
        L.qmm_matmul_f32_workspace_size.restype = sz
        L.qmm_matmul_f32_ws.argtypes = [i32, vp, i64, i64, vp, i64, i64, vp, i64, vp, sz, vp]
        for fn in ("qmm_mx4_codes_size", "qmm_mx4_scales_size", "qmm_mx4_linear_workspace_size"):
            getattr(L, fn).argtypes = [i64, i64]
            getattr(L, fn).restype = sz
        L.qmm_mx4_quantize.argtypes = [i32, vp, i64, i64, i64, vp, vp, vp]
        L.qmm_mx4_dequantize.argtypes = [vp, vp, i64, i64, i32, vp, i64, vp]
        L.qmm_mx4_matmul.argtypes = [vp, vp, i64, i64, vp, vp, i64, i32, vp, i64, vp]
        L.qmm_mx4_linear.argtypes = [vp, vp, i64, i64, i32, vp, i64, i64, i32, vp, i64, vp, sz, vp]
        L.qmm_cache_page_size.argtypes = [i32, i64, i64, i64]
        L.qmm_cache_page_size.restype = sz
        L.qmm_cache_write.argtypes = [i32, i32, vp, vp, i64, i64, i64, i64, i64, vp, vp, vp, i64, i64, vp]
        L.qmm_cache_read.argtypes = [i32, vp, vp, i64, i64, i64, i64, vp, i64, vp, i64, i64, i32, vp, vp, i64, i64, vp]
        L.qmm_cache_attend_workspace_size.argtypes = [i64] * 6
        L.qmm_cache_attend_workspace_size.restype = sz
        L.qmm_cache_attend.argtypes = [i32, vp, vp, i64, i64, i64, i64, vp, i64, vp, vp, i64, i32, vp, i64, i64, i64, vp,
                                       ctypes.c_float, i64, i64, vp, i64, vp, vp, sz, vp]
        for fn in ("qmm_mx4_quantize", "qmm_mx4_dequantize", "qmm_mx4_matmul", "qmm_mx4_linear", "qmm_cache_write",
                   "qmm_cache_read", "qmm_cache_attend", "qmm_quantize_weight", "qmm_repack", "qmm_unpack", "qmm_quantize_act", "qmm_matmul",
                   "qmm_matmul_path", "qmm_device_status", "qmm_matmul_ws", "qmm_matmul_noalloc", "qmm_matmul_f32",
                   "qmm_matmul_flat", "qmm_selftest_timeout", "qmm_matmul_f32_ws"):
            getattr(L, fn).restype = i32
        _lib = L
    return _lib


def _t(type_) -> int:
    return TYPES[type_] if isinstance(type_, str) else int(type_)


def _dt(dtype) -> int:
    return DTYPES[dtype] if isinstance(dtype, str) else int(dtype)


def _ptr(x) -> int | None:
    """Address of a CUDA tensor or of a page-locked (pinned) host tensor, which the GPU reads and
    writes directly (or a raw integer address)."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if not x.is_cuda and not x.is_pinned():
        raise ValueError("libqmm takes CUDA tensors or pinned host tensors only")
    return x.data_ptr()


def _ptr_located(x) -> int | None:
    """Address of a tensor for the calls that check on their own where x and y point (device or
    page-locked host memory; pageable memory is refused by the library): no host-side query here."""
    if x is None or isinstance(x, int):
        return x
    return x.data_ptr()


_raw_stream = None


def _current_stream() -> int:
    """The current stream of the current device as a raw address.  torch's raw queries take a few tenths of a
    microsecond where torch.cuda.current_stream() takes three, half of a small call's host time."""
    global _raw_stream
    if _raw_stream is None:
        import torch

        torch.cuda.current_stream()                                  # initializes CUDA, or says why it cannot
        raw, device = (getattr(torch._C, name, None) for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"))
        _raw_stream = (lambda: raw(device())) if raw and device else (lambda: torch.cuda.current_stream().cuda_stream)
    return _raw_stream()


def _stream(stream) -> int | None:
    if stream is None:
        return _current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(fn: str, st: int) -> None:
    if st != 0:
        raise QmmError(fn, st)


def block_size(type_) -> int:
    return int(lib().qmm_block_size(_t(type_)))


def tile_size(type_) -> int:
    return int(lib().qmm_tile_size(_t(type_)))


def tiled_size(type_, K: int, N: int) -> int:
    return int(lib().qmm_tiled_size(_t(type_), K, N))


def flat_size(type_, K: int, N: int) -> int:
    return int(lib().qmm_flat_size(_t(type_), K, N))


def iq4nl_table() -> list[int]:
    buf = (ctypes.c_int8 * 16)()
    lib().qmm_iq4nl_table(ctypes.cast(buf, ctypes.c_void_p))
    return list(buf)


def decode_max_m() -> int:
    return int(lib().qmm_decode_max_m())


def qmm_quantize_weight(type_, w, N: int, K: int, ldw: int, w_flat, stream=None) -> None:
    _check("qmm_quantize_weight",
           lib().qmm_quantize_weight(_t(type_), _ptr(w), N, K, ldw, _ptr(w_flat), _stream(stream)))


def qmm_repack(type_, w_flat, K: int, N: int, w_tiled, stream=None) -> None:
    _check("qmm_repack", lib().qmm_repack(_t(type_), _ptr(w_flat), K, N, _ptr(w_tiled), _stream(stream)))


def qmm_unpack(type_, w_tiled, K: int, N: int, w_flat, stream=None) -> None:
    _check("qmm_unpack", lib().qmm_unpack(_t(type_), _ptr(w_tiled), K, N, _ptr(w_flat), _stream(stream)))


def qmm_quantize_act(x, M: int, K: int, ldx: int, a_q, a_d, stream=None) -> None:
    _check("qmm_quantize_act",
           lib().qmm_quantize_act(_ptr(x), M, K, ldx, _ptr(a_q), _ptr(a_d), _stream(stream)))


def qmm_matmul(type_, w_tiled, K: int, N: int, a_q, a_d, M: int, y, ldy: int, stream=None) -> None:
    _check("qmm_matmul", lib().qmm_matmul(_t(type_), _ptr(w_tiled), K, N, _ptr(a_q), _ptr(a_d), M, _ptr(y), ldy,
                                          _stream(stream)))


def qmm_matmul_f32(type_, w_tiled, K: int, N: int, x, ldx: int, M: int, y, ldy: int, stream=None) -> None:
    _check("qmm_matmul_f32", lib().qmm_matmul_f32(_t(type_), _ptr(w_tiled), K, N, _ptr_located(x), ldx, M,
                                                  _ptr_located(y), ldy, _stream(stream)))


def matmul_f32_workspace_size(M: int, K: int) -> int:
    return int(lib().qmm_matmul_f32_workspace_size(M, K))


def qmm_matmul_f32_ws(type_, w_tiled, K: int, N: int, x, ldx: int, M: int, y, ldy: int, workspace,
                      workspace_bytes: int, stream=None) -> None:
    _check("qmm_matmul_f32_ws", lib().qmm_matmul_f32_ws(_t(type_), _ptr(w_tiled), K, N, _ptr_located(x), ldx, M,
                                                        _ptr_located(y), ldy, _ptr(workspace), int(workspace_bytes),
                                                        _stream(stream)))


def qmm_matmul_flat(type_, w_flat, K: int, N: int, a_q, a_d, M: int, y, ldy: int, stream=None) -> None:
    _check("qmm_matmul_flat", lib().qmm_matmul_flat(_t(type_), _ptr(w_flat), K, N, _ptr(a_q), _ptr(a_d), M, _ptr(y),
                                                    ldy, _stream(stream)))


def qmm_matmul_path(type_, w_tiled, K: int, N: int, a_q, a_d, M: int, y, ldy: int, path: int,
                    stream=None) -> None:
    _check("qmm_matmul_path", lib().qmm_matmul_path(_t(type_), _ptr(w_tiled), K, N, _ptr(a_q), _ptr(a_d), M,
                                                    _ptr(y), ldy, int(path), _stream(stream)))


def matmul_workspace_size(M: int, K: int) -> int:
    return int(lib().qmm_matmul_workspace_size(M, K))


def qmm_matmul_ws(type_, w_tiled, K: int, N: int, a_q, a_d, M: int, y, ldy: int, workspace, workspace_bytes: int,
                  stream=None) -> None:
    _check("qmm_matmul_ws", lib().qmm_matmul_ws(_t(type_), _ptr(w_tiled), K, N, _ptr(a_q), _ptr(a_d), M, _ptr(y), ldy,
                                                _ptr(workspace), int(workspace_bytes), _stream(stream)))


def qmm_matmul_noalloc(type_, w_tiled, K: int, N: int, a_q, a_d, M: int, y, ldy: int, stream=None) -> None:
    """For callers that cannot allocate device memory: the tensor-core path's workspace is the
    library's fixed per-device scratch array (see include/qmm.h); overlapping calls race on it."""
    _check("qmm_matmul_noalloc", lib().qmm_matmul_noalloc(_t(type_), _ptr(w_tiled), K, N, _ptr(a_q), _ptr(a_d), M,
                                                          _ptr(y), ldy, _stream(stream)))


def matmul_noalloc_max_workspace() -> int:
    return int(lib().qmm_matmul_noalloc_max_workspace())


def qmm_device_status(stream=None) -> int:
    """Synchronize the stream, then return and clear the device status (0 = ok, 5 = timeout)."""
    return int(lib().qmm_device_status(_stream(stream)))


def qmm_selftest_timeout(unit: int, limit_ns: int, flags, stream=None) -> None:
    """Test hook: one CTA whose bounded waits run out on purpose (unit 0: decode kernels' helper,
    1: the GEMM's); afterwards qmm_device_status() reports the timeout (see include/qmm.h)."""
    _check("qmm_selftest_timeout", lib().qmm_selftest_timeout(int(unit), int(limit_ns), _ptr(flags), _stream(stream)))


def mx4_codes_size(R: int, K: int) -> int:
    return int(lib().qmm_mx4_codes_size(R, K))


def mx4_scales_size(R: int, K: int) -> int:
    return int(lib().qmm_mx4_scales_size(R, K))


def mx4_linear_workspace_size(M: int, K: int) -> int:
    return int(lib().qmm_mx4_linear_workspace_size(M, K))


def qmm_mx4_quantize(dtype, x, R: int, K: int, ldx: int, codes, scales, stream=None) -> None:
    """Rows of `dtype` ("f32", "f16", "bf16") -> MX4 operand (codes, scales)."""
    _check("qmm_mx4_quantize", lib().qmm_mx4_quantize(_dt(dtype), _ptr(x), R, K, ldx, _ptr(codes), _ptr(scales), _stream(stream)))


def qmm_mx4_dequantize(codes, scales, R: int, K: int, dtype, y, ldy: int, stream=None) -> None:
    _check("qmm_mx4_dequantize",
           lib().qmm_mx4_dequantize(_ptr(codes), _ptr(scales), R, K, _dt(dtype), _ptr(y), ldy, _stream(stream)))


def qmm_mx4_matmul(w_codes, w_scales, K: int, N: int, a_codes, a_scales, M: int, dtype, y, ldy: int, stream=None) -> None:
    """y[M, N] (of `dtype`) = A @ W^T over MX4 operands."""
    _check("qmm_mx4_matmul", lib().qmm_mx4_matmul(_ptr(w_codes), _ptr(w_scales), K, N, _ptr(a_codes), _ptr(a_scales), M,
                                                  _dt(dtype), _ptr(y), ldy, _stream(stream)))


def qmm_mx4_linear(w_codes, w_scales, K: int, N: int, x_dtype, x, ldx: int, M: int, y_dtype, y, ldy: int, workspace,
                   workspace_bytes: int, stream=None) -> None:
    """y[M, N] = MX4(x) @ W^T: the activations are quantized into the workspace, then multiplied."""
    _check("qmm_mx4_linear", lib().qmm_mx4_linear(_ptr(w_codes), _ptr(w_scales), K, N, _dt(x_dtype), _ptr(x), ldx, M,
                                                  _dt(y_dtype), _ptr(y), ldy, _ptr(workspace), int(workspace_bytes),
                                                  _stream(stream)))


def cache_page_size(type_, H: int, D: int, P: int) -> int:
    return int(lib().qmm_cache_page_size(_t(type_), H, D, P))


def cache_attend_workspace_size(n_seq: int, max_new: int, H: int, Hq: int, D: int, max_len: int) -> int:
    return int(lib().qmm_cache_attend_workspace_size(n_seq, max_new, H, Hq, D, max_len))


def qmm_cache_write(type_, dtype, k, v, ldk: int, ldv: int, T: int, H: int, D: int, slots, k_cache, v_cache, n_pages: int,
                    P: int, stream=None) -> None:
    """Keys and values of T tokens, quantized into their slots (page * P + place) of the paged cache."""
    _check("qmm_cache_write", lib().qmm_cache_write(_t(type_), _dt(dtype), _ptr(k), _ptr(v), ldk, ldv, T, H, D, _ptr(slots),
                                                    _ptr(k_cache), _ptr(v_cache), n_pages, P, _stream(stream)))


def qmm_cache_read(type_, k_cache, v_cache, n_pages: int, P: int, H: int, D: int, pages, ld_pages: int, starts, n_seq: int,
                   T: int, dtype, k, v, ldk: int, ldv: int, stream=None) -> None:
    """The cached values of n_seq sequences as dense rows [T][H][D] of `dtype` (k or v may be None)."""
    _check("qmm_cache_read", lib().qmm_cache_read(_t(type_), _ptr(k_cache), _ptr(v_cache), n_pages, P, H, D, _ptr(pages),
                                                  ld_pages, _ptr(starts), n_seq, T, _dt(dtype), _ptr(k), _ptr(v), ldk, ldv,
                                                  _stream(stream)))


def qmm_cache_attend(type_, k_cache, v_cache, n_pages: int, P: int, H: int, D: int, pages, ld_pages: int, q_starts, kv_lens,
                     n_seq: int, dtype, q, ldq: int, T: int, Hq: int, tree, scale: float, max_new: int, max_len: int, out,
                     ldo: int, lse, workspace, workspace_bytes: int, stream=None) -> None:
    """Attention of each sequence's new tokens (one token, a tree of drafted ones, or a piece of a prompt) over
    its cached tokens; tree, lse and workspace may be None."""
    _check("qmm_cache_attend",
           lib().qmm_cache_attend(_t(type_), _ptr(k_cache), _ptr(v_cache), n_pages, P, H, D, _ptr(pages), ld_pages,
                                  _ptr(q_starts), _ptr(kv_lens), n_seq, _dt(dtype), _ptr(q), ldq, T, Hq, _ptr(tree),
                                  float(scale), max_new, max_len, _ptr(out), ldo, _ptr(lse), _ptr(workspace),
                                  int(workspace_bytes), _stream(stream)))
