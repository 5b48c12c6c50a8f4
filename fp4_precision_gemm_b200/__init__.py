"""Python binding of libfp8q.so (the C ABI declared in include/fp8q.h).

Argument marshalling only: every step of quantization and GEMM runs in the library's CUDA
kernels.  PyTorch supplies device memory (outputs are allocated with torch) and the current
CUDA stream.  There is no CPU fallback: if the library is missing or no CUDA device is
present, the calls raise.

Two layers, same names as the C ABI:
  * ``fp8q_quantize_1x128(...)`` etc. take raw integers/pointers exactly like the C calls;
  * ``quantize_1x128(x, ...)``, ``quantize_128x128``, ``quantize_mx32``, ``quantize_tensor``,
    ``rht16_quantize_sr``, ``gemm`` take torch tensors, allocate the outputs and call them.
"""
import array
import contextlib
import ctypes
import functools
import os

import torch

__all__ = [
    "FP8Q_OK", "FP8Q_BLOCKWISE", "FP8Q_MXFP8", "FP8Q_PERTENSOR", "FP8Q_NVFP4",
    "FP8Q_FPROP", "FP8Q_DGRAD", "FP8Q_WGRAD", "FP8Q_SF_ROWMAJOR", "FP8Q_SF_MMA_TILED",
    "FP4Q_ROW", "FP4Q_COL", "Fp8qError", "lib", "library_path",
    "fp8q_quantize_1x128", "fp8q_quantize_128x128", "fp8q_quantize_mx32", "fp8q_quantize_tensor",
    "fp8q_quantize_tensor_noalloc", "fp8q_quantize_128x128_grouped", "fp8q_quantize_tensor_delayed",
    "fp4q_rht16_quantize_sr", "fp4q_quantize_2d16", "FP8Q_E4M3", "FP8Q_E5M2", "fp8q_gemm_blockscaled", "fp8q_sf_bytes",
    "fp8q_get_device_status", "fp8q_selftest_bounded_wait", "fp8q_status_string", "fp8q_version", "GemmArgs",
    "quantize_1x128", "quantize_128x128", "quantize_128x128_grouped", "quantize_tensor_delayed", "quantize_mx32", "quantize_tensor", "rht16_quantize_sr",
    "quantize_nvfp4_2d16", "gemm", "gemm_workspace_bytes", "device_status", "EXPORTED_SYMBOLS",
    "fp8q_quantize_multi", "fp8q_gemm_workspace_bytes", "QuantItem", "FP8Q_ITEM_1X128", "FP8Q_ITEM_128X128", "FP8Q_MAX_QUANT_ITEMS",
    "quantize_multi", "fp8q_grouped_capacity", "fp8q_quantize_1x128_grouped", "quantize_1x128_grouped",
    "fp8q_clip_grad_norm", "fp8q_clip_grad_workspace_bytes", "GradItem", "clip_grad_norm", "FP8Q_BF16", "FP8Q_FP32",
    "fp8q_norm_residual", "fp8q_norm_residual_backward", "fp8q_norm_backward_workspace_bytes", "NormArgs",
    "NormBackwardArgs", "norm_residual", "norm_residual_backward",
]

FP8Q_OK = 0
FP8Q_ERR_NULL, FP8Q_ERR_SHAPE, FP8Q_ERR_ALIGN, FP8Q_ERR_UNSUPPORTED, FP8Q_ERR_CUDA, FP8Q_ERR_TIMEOUT = 1, 2, 3, 4, 5, 6
FP8Q_ERR_DEVICE_ARG = 7
FP8Q_BLOCKWISE, FP8Q_MXFP8, FP8Q_PERTENSOR, FP8Q_NVFP4 = 0, 1, 2, 3
FP8Q_FPROP, FP8Q_DGRAD, FP8Q_WGRAD = 0, 1, 2
FP8Q_SF_ROWMAJOR, FP8Q_SF_MMA_TILED = 0, 1
FP4Q_ROW, FP4Q_COL = 1, 2
FP8Q_E4M3, FP8Q_E5M2 = 0, 1
FP8Q_ITEM_1X128, FP8Q_ITEM_128X128 = 0, 1
FP8Q_BF16, FP8Q_FP32 = 0, 1
FP8Q_MAX_QUANT_ITEMS = 8

EXPORTED_SYMBOLS = [
    "fp8q_quantize_1x128", "fp8q_quantize_128x128", "fp8q_quantize_mx32", "fp8q_quantize_tensor",
    "fp4q_rht16_quantize_sr", "fp8q_gemm_blockscaled", "fp8q_sf_bytes", "fp8q_get_device_status",
    "fp8q_release_scratch", "fp8q_status_string", "fp8q_version", "fp8q_quantize_tensor_noalloc",
    "fp8q_selftest_bounded_wait", "fp8q_quantize_128x128_grouped", "fp8q_quantize_tensor_delayed",
    "fp4q_quantize_2d16", "fp8q_quantize_multi", "fp8q_gemm_workspace_bytes",
    "fp8q_grouped_capacity", "fp8q_quantize_1x128_grouped",
    "fp8q_clip_grad_norm", "fp8q_clip_grad_workspace_bytes", "fp8q_norm_residual", "fp8q_norm_residual_backward",
    "fp8q_norm_backward_workspace_bytes",
]

library_path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libfp8q.so")
lists_path = os.path.join(os.path.dirname(library_path), "libfp8q_lists.so")


class Fp8qError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        super().__init__(f"{where}: status {status} ({_status_str(status)})")


class QuantItem(ctypes.Structure):
    """Mirror of fp8q_quant_item (field order and types as in include/fp8q.h)."""
    _fields_ = [
        ("kind", ctypes.c_int32), ("x", ctypes.c_void_p),
        ("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("ld_x", ctypes.c_int64),
        ("q_row", ctypes.c_void_p), ("s_row", ctypes.c_void_p), ("ld_s_row", ctypes.c_int64),
        ("q_col", ctypes.c_void_p), ("s_col", ctypes.c_void_p), ("ld_s_col", ctypes.c_int64),
        ("q_t", ctypes.c_void_p), ("q", ctypes.c_void_p), ("s", ctypes.c_void_p),
    ]


class GradItem(ctypes.Structure):
    """Mirror of fp8q_grad_item (field order and types as in include/fp8q.h)."""
    _fields_ = [("grad", ctypes.c_void_p), ("out", ctypes.c_void_p), ("numel", ctypes.c_int64),
                ("dtype", ctypes.c_int64)]


class NormArgs(ctypes.Structure):
    """Mirror of fp8q_norm_args (field order and types as in include/fp8q.h)."""
    _fields_ = [
        ("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("h_dtype", ctypes.c_int32), ("w_dtype", ctypes.c_int32),
        ("alpha", ctypes.c_float), ("eps", ctypes.c_float),
        ("y", ctypes.c_void_p), ("ld_y", ctypes.c_int64), ("h", ctypes.c_void_p), ("ld_h", ctypes.c_int64),
        ("w_post", ctypes.c_void_p), ("gate", ctypes.c_void_p), ("w_pre", ctypes.c_void_p),
        ("h_out", ctypes.c_void_p), ("ld_h_out", ctypes.c_int64), ("n_out", ctypes.c_void_p), ("ld_n", ctypes.c_int64),
        ("q_row", ctypes.c_void_p), ("s_row", ctypes.c_void_p), ("ld_s_row", ctypes.c_int64),
        ("rstd_post", ctypes.c_void_p), ("rstd_pre", ctypes.c_void_p),
    ]


class NormBackwardArgs(ctypes.Structure):
    """Mirror of fp8q_norm_backward_args (field order and types as in include/fp8q.h)."""
    _fields_ = [
        ("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("h_dtype", ctypes.c_int32), ("w_dtype", ctypes.c_int32),
        ("alpha", ctypes.c_float),
        ("dn", ctypes.c_void_p), ("ld_dn", ctypes.c_int64), ("dh_out", ctypes.c_void_p), ("ld_dh_out", ctypes.c_int64),
        ("y", ctypes.c_void_p), ("ld_y", ctypes.c_int64), ("h", ctypes.c_void_p), ("ld_h", ctypes.c_int64),
        ("w_post", ctypes.c_void_p), ("gate", ctypes.c_void_p), ("w_pre", ctypes.c_void_p),
        ("rstd_post", ctypes.c_void_p), ("rstd_pre", ctypes.c_void_p),
        ("dh", ctypes.c_void_p), ("ld_dh", ctypes.c_int64), ("dy", ctypes.c_void_p), ("ld_dy", ctypes.c_int64),
        ("dw_post", ctypes.c_void_p), ("dgate", ctypes.c_void_p), ("dw_pre", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_int64),
    ]


class GemmArgs(ctypes.Structure):
    """Mirror of fp8q_gemm_args (field order and types as in include/fp8q.h)."""
    _fields_ = [
        ("recipe", ctypes.c_int), ("layout", ctypes.c_int),
        ("M", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
        ("a", ctypes.c_void_p), ("a_scale", ctypes.c_void_p), ("lda", ctypes.c_int64), ("ld_sa", ctypes.c_int64),
        ("b", ctypes.c_void_p), ("b_scale", ctypes.c_void_p), ("ldb", ctypes.c_int64), ("ld_sb", ctypes.c_int64),
        ("a_global", ctypes.c_void_p), ("b_global", ctypes.c_void_p),
        ("c", ctypes.c_void_p), ("ldc", ctypes.c_int64),
        ("m_offsets", ctypes.c_void_p), ("num_groups", ctypes.c_int32),
        ("c_fp32_accumulate", ctypes.c_int32),
        ("a_format", ctypes.c_int32), ("b_format", ctypes.c_int32),
        ("q_out", ctypes.c_void_p), ("s_out", ctypes.c_void_p),
        ("ld_q_out", ctypes.c_int64), ("ld_s_out", ctypes.c_int64),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_int64),
    ]


_LIB = None
_i64, _u64, _vp, _int = ctypes.c_int64, ctypes.c_uint64, ctypes.c_void_p, ctypes.c_int


def lib():
    """Loads libfp8q.so once; raises if it has not been built."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(library_path):
            raise ImportError(f"{library_path} is missing: build it with "
                              "`python -m fp4_precision_gemm_b200.build`")
        L = ctypes.CDLL(library_path)
        L.fp8q_quantize_1x128.argtypes = [_vp, _i64, _i64, _i64, _vp, _vp, _i64, _vp, _vp, _i64, _vp]
        L.fp8q_quantize_128x128.argtypes = [_vp, _i64, _i64, _i64, _vp, _vp, _vp, _vp]
        L.fp8q_quantize_128x128_grouped.argtypes = [_vp, _i64, _i64, _i64, _i64, _vp, _vp, _vp, _vp]
        L.fp8q_grouped_capacity.argtypes = [_i64, ctypes.c_int32]
        L.fp8q_grouped_capacity.restype = _i64
        L.fp8q_quantize_1x128_grouped.argtypes = [_vp, _i64, _i64, _i64, _vp, ctypes.c_int32, _vp, _vp, _i64,
                                                  _vp, _vp, _i64, _vp]
        L.fp8q_quantize_mx32.argtypes = [_vp, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _int, _vp]
        L.fp8q_quantize_tensor.argtypes = [_vp, _i64, _i64, _i64, _vp, _vp, _vp]
        L.fp8q_quantize_tensor_noalloc.argtypes = [_vp, _i64, _i64, _i64, _vp, _vp, _vp]
        L.fp8q_quantize_tensor_delayed.argtypes = [_vp, _i64, _i64, _i64, _vp, ctypes.c_int32, ctypes.c_int32, _int,
                                                   _vp, _vp, _vp]
        L.fp4q_rht16_quantize_sr.argtypes = [_vp, _i64, _i64, _i64, _int, _u64, _int, _u64,
                                             _vp, _vp, _vp, _vp, _vp, _vp, _int, _vp]
        L.fp4q_quantize_2d16.argtypes = [_vp, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _int, _vp]
        L.fp8q_gemm_blockscaled.argtypes = [ctypes.POINTER(GemmArgs), _vp]
        L.fp8q_gemm_workspace_bytes.argtypes = [ctypes.POINTER(GemmArgs)]
        L.fp8q_gemm_workspace_bytes.restype = ctypes.c_size_t
        L.fp8q_quantize_multi.argtypes = [ctypes.POINTER(QuantItem), ctypes.c_int32, _vp]
        L.fp8q_norm_residual.argtypes = [ctypes.POINTER(NormArgs), _vp]
        L.fp8q_norm_residual_backward.argtypes = [ctypes.POINTER(NormBackwardArgs), _vp]
        L.fp8q_norm_backward_workspace_bytes.argtypes = [_i64, _i64, ctypes.c_int32]
        L.fp8q_norm_backward_workspace_bytes.restype = ctypes.c_size_t
        L.fp8q_clip_grad_norm.argtypes = [_vp, _i64, ctypes.c_double, ctypes.c_double, _vp, _vp, _i64, _vp]
        L.fp8q_clip_grad_workspace_bytes.argtypes = [_i64]
        L.fp8q_clip_grad_workspace_bytes.restype = ctypes.c_size_t
        L.fp8q_sf_bytes.argtypes = [_int, _i64, _i64, _int]
        L.fp8q_sf_bytes.restype = ctypes.c_size_t
        L.fp8q_get_device_status.argtypes = [_vp]
        L.fp8q_selftest_bounded_wait.argtypes = [_u64, _vp]
        L.fp8q_release_scratch.argtypes = []
        L.fp8q_status_string.argtypes = [_int]
        L.fp8q_status_string.restype = ctypes.c_char_p
        L.fp8q_version.argtypes = []
        L.fp8q_version.restype = ctypes.c_char_p
        for name in EXPORTED_SYMBOLS:
            f = getattr(L, name)
            if f.restype is ctypes.c_int or name in ("fp8q_quantize_1x128", "fp8q_quantize_128x128",
                                                     "fp8q_quantize_mx32", "fp8q_quantize_tensor",
                                                     "fp4q_rht16_quantize_sr", "fp8q_gemm_blockscaled",
                                                     "fp8q_get_device_status", "fp8q_release_scratch",
                                                     "fp8q_selftest_bounded_wait", "fp8q_quantize_128x128_grouped",
                                                     "fp8q_quantize_tensor_delayed", "fp4q_quantize_2d16",
                                                     "fp8q_quantize_multi", "fp8q_quantize_1x128_grouped",
                                                     "fp8q_clip_grad_norm", "fp8q_norm_residual",
                                                     "fp8q_norm_residual_backward"):
                f.restype = ctypes.c_int
        _LIB = L
    return _LIB


_LISTS = None
_DL_CUDA = 2                                               # DLPack's number for CUDA devices


def _lists():
    """The reader of lists of tensors, fp8q_lists_grads with its first three arguments bound; None for a torch
    without the interface that it uses."""
    global _LISTS
    if _LISTS is None:
        if not os.path.exists(lists_path):
            raise ImportError(f"{lists_path} is missing: build it with "
                              "`python -m fp4_precision_gemm_b200.build`")
        L = ctypes.PyDLL(lists_path)
        L.fp8q_lists_api.argtypes, L.fp8q_lists_api.restype = [ctypes.py_object], _vp
        read = L.fp8q_lists_grads
        read.argtypes, read.restype = [_vp] + [ctypes.py_object] * 4 + [ctypes.c_int32, _vp], _i64
        api = L.fp8q_lists_api(getattr(torch.Tensor, "__dlpack_c_exchange_api__", None))
        _LISTS = (None if api is None
                  else functools.partial(read, _vp(api), torch.Tensor, torch.nn.Parameter),)
    return _LISTS[0]


def _status_str(st):
    try:
        return lib().fp8q_status_string(st).decode()
    except Exception:  # noqa: BLE001 - message only
        return "?"


def _check(st, where):
    if st != FP8Q_OK:
        raise Fp8qError(st, where)


def _stream(stream=None):
    if stream is None:
        if not torch.cuda.is_initialized():
            torch.cuda.init()
        try:
            # the handle alone: building a torch.cuda.Stream costs several microseconds a call
            return ctypes.c_void_p(torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice()))
        except AttributeError:                             # a torch without these functions of its own
            stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _current_device():
    try:
        return torch._C._cuda_getDevice()                  # without the public form's checks, 0.2 us a call
    except AttributeError:
        return torch.cuda.current_device()


_HERE = contextlib.nullcontext()


def _on(device, stream):
    """Makes `device`, and `stream` if one is given, current for a call's allocations and launches: memory taken
    for another stream than the one that writes it may still be in use there.  Refuses a stream of another
    device."""
    if stream is not None:
        if stream.device != device:
            raise ValueError(f"stream is on {stream.device}, the tensors are on {device}")
        return torch.cuda.stream(stream)
    index = device.index                                   # None: host tensors, which the checks refuse
    return _HERE if index is None or index == _current_device() else torch.cuda.device(device)


def _results(stream, *made):
    """Tensors that a call made on `stream` (None: the current one) are the caller's to use on the current stream:
    their memory is not given to another call on `stream` before that use has ended."""
    if stream is not None:
        here = torch.cuda.current_stream(stream.device)
        if here != stream:
            for t in made:
                if t is not None:
                    t.record_stream(here)


def _addr(t):
    return None if t is None else t.data_ptr()


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


# --------------------------------------------------------------------------- raw C calls
def fp8q_quantize_1x128(x, rows, cols, ld_x, q_row, s_row, ld_s_row, q_col, s_col, ld_s_col, stream):
    return lib().fp8q_quantize_1x128(x, rows, cols, ld_x, q_row, s_row, ld_s_row, q_col, s_col, ld_s_col, stream)


def fp8q_quantize_128x128(w, K, N, ld_w, q_t, q, s, stream):
    return lib().fp8q_quantize_128x128(w, K, N, ld_w, q_t, q, s, stream)


def fp8q_quantize_multi(items, n_items, stream):
    """items: a ctypes array of QuantItem (or None with n_items == 0)."""
    return lib().fp8q_quantize_multi(items, n_items, stream)


def fp8q_quantize_128x128_grouped(w, groups, K, N, ld_w, q_t, q, s, stream):
    return lib().fp8q_quantize_128x128_grouped(w, groups, K, N, ld_w, q_t, q, s, stream)


def fp8q_grouped_capacity(rows, groups):
    return int(lib().fp8q_grouped_capacity(rows, groups))


def fp8q_quantize_1x128_grouped(x, rows, cols, ld_x, offsets, groups, q_row, s_row, ld_s_row, q_col, s_col, ld_s_col,
                                stream):
    return lib().fp8q_quantize_1x128_grouped(x, rows, cols, ld_x, offsets, groups, q_row, s_row, ld_s_row, q_col,
                                             s_col, ld_s_col, stream)


def fp8q_quantize_mx32(x, rows, cols, ld_x, q_row, e_row, q_col, e_col, sf_layout, stream):
    return lib().fp8q_quantize_mx32(x, rows, cols, ld_x, q_row, e_row, q_col, e_col, sf_layout, stream)


def fp8q_quantize_tensor(x, rows, cols, ld_x, q, s_dec, stream):
    return lib().fp8q_quantize_tensor(x, rows, cols, ld_x, q, s_dec, stream)


def fp8q_quantize_tensor_delayed(x, rows, cols, ld_x, hist, hlen, hpos, fmt, q, s_dec, stream):
    return lib().fp8q_quantize_tensor_delayed(x, rows, cols, ld_x, hist, hlen, hpos, fmt, q, s_dec, stream)


def fp8q_quantize_tensor_noalloc(x, rows, cols, ld_x, q, s_dec, stream):
    """Per-tensor quantization that allocates no device memory (scratch in the library's
    fixed device array); for callers that cannot let a library allocate."""
    return lib().fp8q_quantize_tensor_noalloc(x, rows, cols, ld_x, q, s_dec, stream)


def fp4q_rht16_quantize_sr(x, rows, cols, ld_x, rht, rht_seed, sr, sr_seed, q_row, sf_row, g_row,
                           q_col, sf_col, g_col, sf_layout, stream):
    return lib().fp4q_rht16_quantize_sr(x, rows, cols, ld_x, rht, rht_seed, sr, sr_seed, q_row, sf_row, g_row,
                                        q_col, sf_col, g_col, sf_layout, stream)


def fp4q_quantize_2d16(x, rows, cols, ld_x, q_row, sf_row, q_col, sf_col, g_dec, sf_layout, stream):
    return lib().fp4q_quantize_2d16(x, rows, cols, ld_x, q_row, sf_row, q_col, sf_col, g_dec, sf_layout, stream)


def fp8q_gemm_blockscaled(args, stream):
    return lib().fp8q_gemm_blockscaled(ctypes.byref(args), stream)


def fp8q_gemm_workspace_bytes(args):
    return lib().fp8q_gemm_workspace_bytes(ctypes.byref(args))


def fp8q_norm_residual(args, stream):
    return lib().fp8q_norm_residual(ctypes.byref(args), stream)


def fp8q_norm_residual_backward(args, stream):
    return lib().fp8q_norm_residual_backward(ctypes.byref(args), stream)


def fp8q_norm_backward_workspace_bytes(rows, cols, h_dtype):
    return int(lib().fp8q_norm_backward_workspace_bytes(rows, cols, h_dtype))


def fp8q_clip_grad_norm(items, n_items, max_norm, eps, norm, workspace, workspace_bytes, stream):
    """items: a ctypes array of GradItem or its address (or None with n_items == 0)."""
    return lib().fp8q_clip_grad_norm(items, n_items, max_norm, eps, norm, workspace, workspace_bytes, stream)


def fp8q_clip_grad_workspace_bytes(n_items):
    return int(lib().fp8q_clip_grad_workspace_bytes(n_items))


def fp8q_sf_bytes(recipe, outer, inner, layout):
    return int(lib().fp8q_sf_bytes(recipe, outer, inner, layout))


def fp8q_get_device_status(stream):
    return lib().fp8q_get_device_status(stream)


def fp8q_selftest_bounded_wait(limit_ns, stream):
    return lib().fp8q_selftest_bounded_wait(limit_ns, stream)


def fp8q_status_string(st):
    return lib().fp8q_status_string(st).decode()


def fp8q_version():
    return lib().fp8q_version().decode()


# --------------------------------------------------------------------------- tensor API
def _check_bf16(x, name="x"):
    if not (x.is_cuda and x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1):
        raise ValueError(f"{name} must be a 2-D row-major CUDA bf16 tensor")


def quantize_1x128(x, rowwise=True, colwise=False, stream=None):
    """1x128 tiles.  Returns dict with q_row (R, C) uint8, s_row (C/128, R) float32 and/or
    q_col (C, R) uint8, s_col (R/128, C) float32."""
    _check_bf16(x)
    R, C = x.shape
    with _on(x.device, stream):
        out = {}
        if rowwise:
            out["q_row"] = x.new_empty((R, C), dtype=torch.uint8)
            out["s_row"] = x.new_empty((C // 128, max(R, 1) + (-max(R, 1)) % 4), dtype=torch.float32)
        if colwise:
            out["q_col"] = x.new_empty((C, R), dtype=torch.uint8)
            out["s_col"] = x.new_empty((R // 128, C + (-C) % 4), dtype=torch.float32)
        st = fp8q_quantize_1x128(_ptr(x), R, C, x.stride(0), _ptr(out.get("q_row")), _ptr(out.get("s_row")),
                                 out["s_row"].shape[1] if rowwise else 0, _ptr(out.get("q_col")),
                                 _ptr(out.get("s_col")), out["s_col"].shape[1] if colwise else 0, _stream())
    _check(st, "fp8q_quantize_1x128")
    _results(stream, *out.values())
    return out


def quantize_128x128(w, transposed=True, plain=True, stream=None):
    """128x128 blocks of W (K x N).  Returns q_t (N, K), q (K, N), s (N/128, K/128)."""
    _check_bf16(w, "w")
    K, N = w.shape
    with _on(w.device, stream):
        out = {"s": w.new_empty((N // 128, K // 128), dtype=torch.float32)}
        if transposed:
            out["q_t"] = w.new_empty((N, K), dtype=torch.uint8)
        if plain:
            out["q"] = w.new_empty((K, N), dtype=torch.uint8)
        st = fp8q_quantize_128x128(_ptr(w), K, N, w.stride(0), _ptr(out.get("q_t")), _ptr(out.get("q")),
                                   _ptr(out["s"]), _stream())
    _check(st, "fp8q_quantize_128x128")
    _results(stream, *out.values())
    return out


def quantize_multi(specs, stream=None):
    """Several quantizations in one launch.  specs: a list of ("1x128", x, rowwise, colwise)
    and ("128x128", w, transposed, plain) tuples.  Returns one output dict per spec, laid
    out exactly as quantize_1x128 / quantize_128x128 return them."""
    with _on(specs[0][1].device, stream) if specs else _HERE:
        items = (QuantItem * max(len(specs), 1))()
        outs = []
        n = 0
        for spec in specs:
            kind, x, a, b = spec
            _check_bf16(x)
            R, C = x.shape
            it = items[n] if x.numel() else QuantItem()   # an empty tensor has nothing to launch
            n += 1 if x.numel() else 0
            it.x, it.rows, it.cols, it.ld_x = x.data_ptr(), R, C, x.stride(0)
            out = {}
            if kind == "1x128":
                it.kind = FP8Q_ITEM_1X128
                if a:
                    out["q_row"] = x.new_empty((R, C), dtype=torch.uint8)
                    out["s_row"] = x.new_empty((C // 128, max(R, 1) + (-max(R, 1)) % 4), dtype=torch.float32)
                    it.q_row, it.s_row, it.ld_s_row = out["q_row"].data_ptr(), out["s_row"].data_ptr(), out["s_row"].shape[1]
                if b:
                    out["q_col"] = x.new_empty((C, R), dtype=torch.uint8)
                    out["s_col"] = x.new_empty((R // 128, C + (-C) % 4), dtype=torch.float32)
                    it.q_col, it.s_col, it.ld_s_col = out["q_col"].data_ptr(), out["s_col"].data_ptr(), out["s_col"].shape[1]
            elif kind == "128x128":
                it.kind = FP8Q_ITEM_128X128
                out["s"] = x.new_empty((C // 128, R // 128), dtype=torch.float32)
                it.s = out["s"].data_ptr()
                if a:
                    out["q_t"] = x.new_empty((C, R), dtype=torch.uint8)
                    it.q_t = out["q_t"].data_ptr()
                if b:
                    out["q"] = x.new_empty((R, C), dtype=torch.uint8)
                    it.q = out["q"].data_ptr()
            else:
                raise ValueError(f"unknown quantization kind {kind!r}")
            outs.append(out)
        st = fp8q_quantize_multi(items, n, _stream())
    _check(st, "fp8q_quantize_multi")
    for out in outs:
        _results(stream, *out.values())
    return outs


def quantize_128x128_grouped(w, transposed=True, plain=True, stream=None):
    """128x128 blocks of every matrix of a stack W (G x K x N, contiguous matrices) in one
    call.  Returns q_t (G, N, K), q (G, K, N), s (G, N/128, K/128)."""
    if w.dim() != 3 or w.dtype != torch.bfloat16 or not w.is_cuda:
        raise ValueError("w must be a CUDA bfloat16 tensor of shape (G, K, N)")
    if w.stride(2) != 1 or w.stride(0) != w.shape[1] * w.stride(1):
        raise ValueError("w must hold contiguous row-major matrices (row stride may be padded)")
    G, K, N = w.shape
    with _on(w.device, stream):
        out = {"s": w.new_empty((G, N // 128, K // 128), dtype=torch.float32)}
        if transposed:
            out["q_t"] = w.new_empty((G, N, K), dtype=torch.uint8)
        if plain:
            out["q"] = w.new_empty((G, K, N), dtype=torch.uint8)
        st = fp8q_quantize_128x128_grouped(_ptr(w), G, K, N, w.stride(1), _ptr(out.get("q_t")), _ptr(out.get("q")),
                                           _ptr(out["s"]), _stream())
    _check(st, "fp8q_quantize_128x128_grouped")
    _results(stream, *out.values())
    return out


def _check_offsets(m_offsets, device):
    if not (m_offsets.device == device and m_offsets.dtype == torch.int32 and m_offsets.is_contiguous()
            and m_offsets.numel() >= 2):
        raise ValueError("m_offsets must be a contiguous int32 tensor of groups + 1 offsets on the operands' device")


def quantize_1x128_grouped(x, m_offsets, rowwise=False, colwise=True, stream=None):
    """1x128 tiles of routed tokens x (R, C), expert g's being rows m_offsets[g] .. m_offsets[g + 1] - 1 (int32
    CUDA tensor of groups + 1), with no tile over two experts' tokens.  Returns q_col (C, P) uint8, s_col
    (P/128, C) float32 on the padded token axis P = fp8q_grouped_capacity(R, groups), the grouped WGRAD operands
    of gemm(), and with rowwise q_row (R, C), s_row (C/128, R) as quantize_1x128 returns them."""
    _check_bf16(x)
    _check_offsets(m_offsets, x.device)
    if not colwise:
        raise ValueError("grouping only concerns the colwise output: use quantize_1x128 for rowwise alone")
    R, C = x.shape
    groups = m_offsets.numel() - 1
    P = fp8q_grouped_capacity(R, groups)
    with _on(x.device, stream):
        out = {"q_col": x.new_empty((C, P), dtype=torch.uint8),
               "s_col": x.new_empty((P // 128, C + (-C) % 4), dtype=torch.float32)}
        if rowwise:
            out["q_row"] = x.new_empty((R, C), dtype=torch.uint8)
            out["s_row"] = x.new_empty((C // 128, max(R, 1) + (-max(R, 1)) % 4), dtype=torch.float32)
        st = fp8q_quantize_1x128_grouped(_ptr(x), R, C, x.stride(0), _ptr(m_offsets), groups, _ptr(out.get("q_row")),
                                         _ptr(out.get("s_row")), out["s_row"].shape[1] if rowwise else 0,
                                         _ptr(out["q_col"]), _ptr(out["s_col"]), out["s_col"].shape[1], _stream())
    _check(st, "fp8q_quantize_1x128_grouped")
    _results(stream, *out.values())
    return out


def quantize_mx32(x, rowwise=True, colwise=False, sf_layout=FP8Q_SF_ROWMAJOR, stream=None):
    """MXFP8.  Returns q_row (R, C) + e8m0_row, and/or q_col (C, R) + e8m0_col (flat uint8
    buffers sized by fp8q_sf_bytes for the chosen layout)."""
    _check_bf16(x)
    R, C = x.shape
    with _on(x.device, stream):
        out = {}
        if rowwise:
            out["q_row"] = x.new_empty((R, C), dtype=torch.uint8)
            out["e8m0_row"] = x.new_empty(fp8q_sf_bytes(FP8Q_MXFP8, R, C, sf_layout), dtype=torch.uint8)
        if colwise:
            out["q_col"] = x.new_empty((C, R), dtype=torch.uint8)
            out["e8m0_col"] = x.new_empty(fp8q_sf_bytes(FP8Q_MXFP8, C, R, sf_layout), dtype=torch.uint8)
        st = fp8q_quantize_mx32(_ptr(x), R, C, x.stride(0), _ptr(out.get("q_row")), _ptr(out.get("e8m0_row")),
                                _ptr(out.get("q_col")), _ptr(out.get("e8m0_col")), sf_layout, _stream())
    _check(st, "fp8q_quantize_mx32")
    _results(stream, *out.values())
    return out


def quantize_tensor(x, stream=None):
    """Per-tensor current scaling.  Returns q (R, C) uint8 and s_dec (1,) float32."""
    _check_bf16(x)
    R, C = x.shape
    with _on(x.device, stream):
        out = {"q": x.new_empty((R, C), dtype=torch.uint8),
               "s_dec": x.new_empty((1,), dtype=torch.float32)}
        st = fp8q_quantize_tensor(_ptr(x), R, C, x.stride(0), _ptr(out["q"]), _ptr(out["s_dec"]), _stream())
    _check(st, "fp8q_quantize_tensor")
    _results(stream, *out.values())
    return out


def quantize_tensor_delayed(x, amax_history, history_pos, fmt=FP8Q_E4M3, stream=None):
    """Per-tensor delayed scaling: scale from max(amax_history) (float32 CUDA tensor, updated
    in place at history_pos with this tensor's amax).  Returns q (R, C) uint8, s_dec (1,)."""
    _check_bf16(x)
    if not (amax_history.is_cuda and amax_history.dtype == torch.float32 and amax_history.dim() == 1):
        raise ValueError("amax_history must be a 1-D float32 CUDA tensor")
    R, C = x.shape
    with _on(x.device, stream):
        out = {"q": x.new_empty((R, C), dtype=torch.uint8),
               "s_dec": x.new_empty((1,), dtype=torch.float32)}
        st = fp8q_quantize_tensor_delayed(_ptr(x), R, C, x.stride(0), _ptr(amax_history), amax_history.numel(),
                                          history_pos, fmt, _ptr(out["q"]), _ptr(out["s_dec"]), _stream())
    _check(st, "fp8q_quantize_tensor_delayed")
    _results(stream, *out.values())
    return out


def rht16_quantize_sr(x, rowwise=True, colwise=False, rht=0, rht_seed=0, sr=0, sr_seed=0,
                      sf_layout=FP8Q_SF_ROWMAJOR, stream=None):
    """NVFP4.  rht / sr are FP4Q_ROW | FP4Q_COL masks.  Returns q_row (R, C/2), sf_row,
    g_row (1,) and/or q_col (C, R/2), sf_col, g_col (1,)."""
    _check_bf16(x)
    R, C = x.shape
    with _on(x.device, stream):
        out = {}
        if rowwise:
            out["q_row"] = x.new_empty((R, C // 2), dtype=torch.uint8)
            out["sf_row"] = x.new_empty(fp8q_sf_bytes(FP8Q_NVFP4, R, C, sf_layout), dtype=torch.uint8)
            out["g_row"] = x.new_empty((1,), dtype=torch.float32)
        if colwise:
            out["q_col"] = x.new_empty((C, R // 2), dtype=torch.uint8)
            out["sf_col"] = x.new_empty(fp8q_sf_bytes(FP8Q_NVFP4, C, R, sf_layout), dtype=torch.uint8)
            out["g_col"] = x.new_empty((1,), dtype=torch.float32)
        st = fp4q_rht16_quantize_sr(_ptr(x), R, C, x.stride(0), rht, rht_seed, sr, sr_seed,
                                    _ptr(out.get("q_row")), _ptr(out.get("sf_row")), _ptr(out.get("g_row")),
                                    _ptr(out.get("q_col")), _ptr(out.get("sf_col")), _ptr(out.get("g_col")),
                                    sf_layout, _stream())
    _check(st, "fp4q_rht16_quantize_sr")
    _results(stream, *out.values())
    return out


def quantize_nvfp4_2d16(w, rowwise=True, colwise=True, sf_layout=FP8Q_SF_MMA_TILED, stream=None):
    """NVFP4 weights with one scale per 16x16 block.  Returns q_row (R, C/2), sf_row and/or
    q_col (C, R/2), sf_col, and g (1,), the decode scale both layouts share."""
    _check_bf16(w, "w")
    R, C = w.shape
    with _on(w.device, stream):
        out = {"g": w.new_empty((1,), dtype=torch.float32)}
        if rowwise:
            out["q_row"] = w.new_empty((R, C // 2), dtype=torch.uint8)
            out["sf_row"] = w.new_empty(fp8q_sf_bytes(FP8Q_NVFP4, R, C, sf_layout), dtype=torch.uint8)
        if colwise:
            out["q_col"] = w.new_empty((C, R // 2), dtype=torch.uint8)
            out["sf_col"] = w.new_empty(fp8q_sf_bytes(FP8Q_NVFP4, C, R, sf_layout), dtype=torch.uint8)
        st = fp4q_quantize_2d16(_ptr(w), R, C, w.stride(0), _ptr(out.get("q_row")), _ptr(out.get("sf_row")),
                                _ptr(out.get("q_col")), _ptr(out.get("sf_col")), _ptr(out["g"]), sf_layout,
                                _stream())
    _check(st, "fp4q_quantize_2d16")
    _results(stream, *out.values())
    return out


_CODES = (torch.uint8, torch.int8, torch.float8_e4m3fn)       # E4M3 codes, by any of their types


def _check_scales(name, t, ld, rows, cols, experts=1):
    """Checks that t holds `experts` times `rows` rows of `cols` scales, every row `ld` after the one before it; ld
    None: t is contiguous and its last dimension is ld."""
    if t is None:
        return
    shape, n = t.shape, experts * rows
    if ld is not None:                                             # what t spans, from its first element to its last
        span = 1 + sum((k - 1) * s for k, s in zip(shape, t.stride())) if t.numel() else 0
    else:
        ld, span = shape[-1] if len(shape) > 1 else 0, t.numel()
        # experts in a dimension of their own must also be `rows` rows apart
        if not t.is_contiguous() or (experts > 1 and len(shape) > 2 and shape[0] > 1 and span != shape[0] * rows * ld):
            span = -1
    if t.dtype is not torch.float32 or ld < cols or span < 0 or (n and (n - 1) * ld + cols > span):
        raise ValueError(f"{name} must be float32 and hold {experts} x {rows} rows of {cols}: contiguous, or its "
                         f"leading dimension given")


def _check_grouped(a, b, layout, a_scale, b_scale, ld_sa, ld_sb, K, m_offsets, out, accumulate_fp32):
    """Checks the tensors of a grouped gemm() (the kernels read whole tiles at the strides they are given: a wrong
    shape would read past its tensor) for what the kernels read and write of them; returns the number of experts,
    K and C's shape."""
    _check_offsets(m_offsets, a.device)
    index = a.get_device()
    for t in (b, a_scale, b_scale, out):
        if t is not None and t.get_device() != index:
            raise ValueError("grouped operands must be on one device")
    groups, k_groups = m_offsets.numel() - 1, layout == FP8Q_WGRAD        # WGRAD: experts split K; C is stacked
    a_shape, b_shape, b_strides = a.shape, b.shape, b.stride()
    if len(b_shape) != (2 if k_groups else 3) or len(a_shape) != 2:
        raise ValueError("grouped b must be (G, N, K) codes, or (N, P) on the padded token axis for WGRAD")
    if a.dtype not in _CODES or b.dtype not in _CODES or a.stride(1) != 1 or b_strides[-1] != 1:
        raise ValueError("grouped a and b must be row-major uint8 (or E4M3) codes")
    (M, a_cols), (N, b_cols) = a_shape, b_shape[-2:]
    if K is None:
        K = a_cols
        if b_cols < K:
            raise ValueError("a and b must have the same K")
    elif not 0 <= K <= min(a_cols, b_cols):
        raise ValueError(f"K must be between 0 and the columns of a and b: {K}, {a_cols}, {b_cols}")
    if not k_groups and (b_shape[0] < groups or (groups > 1 and b_strides[0] != N * b_strides[1])):
        raise ValueError("b must hold one matrix per expert, one directly after the other")
    kb, nb = -(-K // 128), -(-N // 128)
    _check_scales("a_scale", a_scale, ld_sa, kb, M)
    if k_groups:
        _check_scales("b_scale", b_scale, ld_sb, kb, N)
    elif layout == FP8Q_DGRAD:
        _check_scales("b_scale", b_scale, ld_sb, kb, nb, groups)
    else:
        _check_scales("b_scale", b_scale, ld_sb, nb, kb, groups)
    shape = (groups, M, N) if k_groups else (M, N)
    if out is not None:
        if out.dtype is not (torch.float32 if accumulate_fp32 else torch.bfloat16) or out.stride(-1) != 1:
            raise ValueError(f"grouped `out` must be row-major {shape}, bfloat16 or, with accumulate_fp32, float32")
        if k_groups:
            if out.shape != shape or (groups > 1 and out.stride(0) != M * out.stride(1)):
                raise ValueError(f"grouped WGRAD `out` must be {shape}, one matrix directly after the other")
        elif out.dim() != 2 or out.shape[0] < M or out.shape[1] < N:
            raise ValueError(f"grouped `out` must have {M} rows and {N} columns, or more")
    if index < 0:
        raise ValueError("grouped a, b, a_scale, b_scale and `out` must be on a CUDA device")
    return groups, K, shape


def _gemm_args(a, b, recipe, layout, a_scale, b_scale, ld_sa, ld_sb, a_global, b_global, K, m_offsets, out,
               accumulate_fp32, a_format, b_format, q_out, s_out):
    """The C ABI's argument block for gemm() (and the output tensor it writes)."""
    M, N = a.shape[0], b.shape[-2]
    if accumulate_fp32 and (out is None or out.dtype != torch.float32):
        raise ValueError("accumulate_fp32 needs an FP32 `out` tensor to update")
    groups, shape = 0, (M, N)
    if m_offsets is None:
        index = a.get_device()
        if index < 0 or b.get_device() != index:
            raise ValueError("operands must be on one CUDA device")
        for t in (a_scale, b_scale, a_global, b_global, out, q_out, s_out):
            if t is not None and t.get_device() != index:
                raise ValueError("operands must be on one CUDA device")
    else:
        groups, K, shape = _check_grouped(a, b, layout, a_scale, b_scale, ld_sa, ld_sb, K, m_offsets, out,
                                          accumulate_fp32)
    if K is None:
        K = a.shape[1] * (2 if recipe == FP8Q_NVFP4 else 1)
    c = out if out is not None else a.new_empty(shape, dtype=torch.bfloat16)
    if ld_sa is None:
        ld_sa = a_scale.shape[-1] if (a_scale is not None and a_scale.dim() == 2) else 0
    if ld_sb is None:
        ld_sb = b_scale.shape[-1] if (b_scale is not None and b_scale.dim() >= 2) else 0
    args = GemmArgs(recipe, layout, M, N, K, a.data_ptr(), _addr(a_scale), a.stride(0), ld_sa, b.data_ptr(),
                    _addr(b_scale), b.stride(-2), ld_sb, _addr(a_global), _addr(b_global), c.data_ptr(), c.stride(-2),
                    _addr(m_offsets), groups, 1 if accumulate_fp32 else 0, a_format, b_format)
    if q_out is not None or s_out is not None:
        args.q_out = q_out.data_ptr() if q_out is not None else None
        args.s_out = s_out.data_ptr() if s_out is not None else None
        args.ld_q_out = q_out.stride(0) if q_out is not None else 0
        args.ld_s_out = s_out.stride(0) if s_out is not None else 0
    return args, c


def gemm(a, b, recipe=FP8Q_BLOCKWISE, layout=FP8Q_FPROP, a_scale=None, b_scale=None, ld_sa=None, ld_sb=None,
         a_global=None, b_global=None, K=None, m_offsets=None, out=None, accumulate_fp32=False,
         a_format=0, b_format=0, q_out=None, s_out=None, stream=None, split_tail=True):
    """C = A . B^T (BF16).  a: (M, K or K/2) uint8 codes, b: (N, ...) or (G, N, ...) uint8.
    Scales as the C ABI describes for the recipe.  Returns C (M, N) bf16.
    m_offsets (BLOCKWISE; int32 CUDA tensor of G + 1): products grouped by expert.  FPROP and DGRAD: expert g's
    rows of a and C are m_offsets[g] .. m_offsets[g + 1] - 1, b is (G, N, K) and b_scale stacked likewise.
    WGRAD: a (M, P) and b (N, P) are quantize_1x128_grouped's colwise codes for the same offsets, and C is
    (G, M, N), expert g's product running over its own tokens only.
    accumulate_fp32 (BLOCKWISE): `out` is an FP32 (M, N) tensor updated in place, C += A . B^T.
    q_out (M, N) uint8 and s_out (N/128, M) float32 (BLOCKWISE): also receive the 1x128
    rowwise quantization of the BF16 C, made in the GEMM's epilogue.
    split_tail (BLOCKWISE, not grouped, no q_out): give the call the workspace it asks for
    (fp8q_gemm_workspace_bytes), taken from torch's caching allocator on the call's stream, so
    that a mostly idle last wave is split into K ranges."""
    with _on(a.device, stream):
        args, c = _gemm_args(a, b, recipe, layout, a_scale, b_scale, ld_sa, ld_sb, a_global, b_global, K, m_offsets,
                             out, accumulate_fp32, a_format, b_format, q_out, s_out)
        if split_tail and recipe == FP8Q_BLOCKWISE and m_offsets is None:
            nbytes = fp8q_gemm_workspace_bytes(args)
            if nbytes > 0:
                ws = a.new_empty((nbytes,), dtype=torch.uint8)
                args.workspace, args.workspace_bytes = ws.data_ptr(), nbytes
        _check(fp8q_gemm_blockscaled(args, _stream()), "fp8q_gemm_blockscaled")
    _results(stream, c if out is None else None)
    return c


def gemm_workspace_bytes(M, N, K, recipe=FP8Q_BLOCKWISE, layout=FP8Q_FPROP, accumulate_fp32=False,
                         fused_quant=False, grouped=False):
    """Workspace bytes gemm() gives a call of this kind and size (0: the call launches one
    kernel; otherwise two: the tiles with the last wave's K ranges, then the sum of the ranges)."""
    args = GemmArgs()
    args.recipe, args.layout = recipe, layout
    args.M, args.N, args.K = M, N, K
    args.c_fp32_accumulate = 1 if accumulate_fp32 else 0
    args.num_groups = 1 if grouped else 0
    if fused_quant:
        args.q_out, args.s_out = 16, 16          # only their presence is read
    return fp8q_gemm_workspace_bytes(args)


_DTYPES = {torch.bfloat16: FP8Q_BF16, torch.float32: FP8Q_FP32}


def _matrix(t, dtype, shape, index):
    """Checks a norm call's matrix; returns its row stride (a single row has the columns': its own means nothing)."""
    strides = t.stride()
    if t.dtype is not dtype or t.shape != shape or t.get_device() != index or strides[1] != 1:
        raise ValueError(f"matrices must be row-major, of y's shape and on its device; this one must be {dtype}")
    return strides[0] if shape[0] > 1 else shape[1]


def _vector(t, dtype, n, index):
    if (t.dtype is not dtype or t.get_device() != index or t.dim() != 1 or t.numel() != n
            or not t.is_contiguous()):
        raise ValueError(f"expected a contiguous {dtype} vector of {n} on y's device")
    return t.data_ptr()


def norm_residual(y, h, w_pre, w_post=None, gate=None, alpha=1.0, eps=1e-6, normed=True, quantize=False, out=None,
                  stream=None):
    """h' = alpha h + gate * norm(y) * w_post (without w_post: the plain y; without gate: 1) and the next block's
    norm n = norm(h') * w_pre, RMS norms over the columns, in one pass.  y (R, C) bfloat16; h (R, C) bfloat16 or
    float32; w_pre, w_post, gate (C,) bfloat16 or float32, all of one type.  Returns h (h', h's type; written to
    `out` if given, which may be h itself), n (R, C) bfloat16 if `normed`, q_row and s_row (the 1x128
    quantization of n, laid out as quantize_1x128 does) if `quantize`, and rstd_pre, rstd_post (R,) float32 for
    norm_residual_backward (rstd_post None without w_post)."""
    _check_bf16(y, "y")
    shape, index, dev, hd, wd = y.shape, y.get_device(), y.device, h.dtype, w_pre.dtype
    R, C = shape
    if hd not in _DTYPES or wd not in _DTYPES:
        raise ValueError("h and the weights must be bfloat16 or float32")
    if not (normed or quantize):
        raise ValueError("neither output of the norm is asked for")
    ld_y, ld_h = _matrix(y, torch.bfloat16, shape, index), _matrix(h, hd, shape, index)
    p_pre = _vector(w_pre, wd, C, index)
    p_post = None if w_post is None else _vector(w_post, wd, C, index)
    p_gate = None if gate is None else _vector(gate, wd, C, index)
    with _on(dev, stream):
        own = None
        if out is None:
            own = out = torch.empty_like(h, memory_format=torch.contiguous_format)
            ld_out = C
        else:
            ld_out = _matrix(out, hd, shape, index)
        rstd = y.new_empty((R,), dtype=torch.float32)
        rstd_post = None if w_post is None else y.new_empty((R,), dtype=torch.float32)
        o = {"h": out, "rstd_pre": rstd, "rstd_post": rstd_post}
        n = q = sc = None
        ld_s = 0
        if normed:
            o["n"] = n = torch.empty_like(y, memory_format=torch.contiguous_format)
        if quantize:
            ld_s = max(R, 1) + (-max(R, 1)) % 4
            o["q_row"] = q = torch.empty_like(y, dtype=torch.uint8, memory_format=torch.contiguous_format)
            o["s_row"] = sc = y.new_empty((C // 128, ld_s), dtype=torch.float32)
        a = NormArgs(R, C, _DTYPES[hd], _DTYPES[wd], alpha, eps, y.data_ptr(), ld_y, h.data_ptr(), ld_h, p_post, p_gate,
                     p_pre, out.data_ptr(), ld_out, _addr(n), C, _addr(q), _addr(sc), ld_s, _addr(rstd_post),
                     rstd.data_ptr())
        _check(fp8q_norm_residual(a, _stream()), "fp8q_norm_residual")
    _results(stream, own, rstd, rstd_post, n, q, sc)
    return o


def norm_residual_backward(dn, dh, y, h, rstd_pre, w_pre, w_post=None, rstd_post=None, gate=None, alpha=1.0,
                           stream=None):
    """Gradients of norm_residual from dn (of n, bfloat16) and dh (of h', of h's type); y, w_pre, w_post, gate and
    alpha as given to it, h, rstd_pre and rstd_post as it returned them.  Returns dh (of the incoming residual),
    dy (bfloat16), and float32 dw_pre, with w_post dw_post, with gate dgate (C,)."""
    _check_bf16(y, "y")
    shape, index, dev, hd, wd = y.shape, y.get_device(), y.device, h.dtype, w_pre.dtype
    R, C = shape
    if hd not in _DTYPES or wd not in _DTYPES:
        raise ValueError("h and the weights must be bfloat16 or float32")
    if (w_post is None) != (rstd_post is None):
        raise ValueError("w_post and rstd_post go together")
    ld_dn, ld_y = _matrix(dn, torch.bfloat16, shape, index), _matrix(y, torch.bfloat16, shape, index)
    ld_dh, ld_h = _matrix(dh, hd, shape, index), _matrix(h, hd, shape, index)
    p_rstd, p_pre = _vector(rstd_pre, torch.float32, R, index), _vector(w_pre, wd, C, index)
    p_post = p_rstd_post = p_gate = None
    names = ["dw_pre"]
    if w_post is not None:
        p_post, p_rstd_post = _vector(w_post, wd, C, index), _vector(rstd_post, torch.float32, R, index)
        names.append("dw_post")
    if gate is not None:
        p_gate = _vector(gate, wd, C, index)
        names.append("dgate")
    with _on(dev, stream):
        dh_in = torch.empty_like(h, memory_format=torch.contiguous_format)
        dy = torch.empty_like(y, memory_format=torch.contiguous_format)
        sums = y.new_empty((len(names), C), dtype=torch.float32)      # one allocation for the vectors
        o = {"dh": dh_in, "dy": dy, **dict(zip(names, sums.unbind(0)))}
        at = dict(zip(names, range(sums.data_ptr(), sums.data_ptr() + 4 * C * len(names), 4 * C)))
        nbytes = fp8q_norm_backward_workspace_bytes(R, C, _DTYPES[hd])
        ws = y.new_empty((max(nbytes, 16),), dtype=torch.uint8)
        a = NormBackwardArgs(R, C, _DTYPES[hd], _DTYPES[wd], alpha, dn.data_ptr(), ld_dn, dh.data_ptr(), ld_dh,
                             y.data_ptr(), ld_y, h.data_ptr(), ld_h, p_post, p_gate, p_pre, p_rstd_post, p_rstd,
                             dh_in.data_ptr(), C, dy.data_ptr(), C, at.get("dw_post"), at.get("dgate"), at["dw_pre"],
                             ws.data_ptr(), nbytes)
        _check(fp8q_norm_residual_backward(a, _stream()), "fp8q_norm_residual_backward")
    _results(stream, dh_in, dy, sums)
    return o


def _grad_items(grads, outs):
    """The C call's items (an object with their memory, and its address) for a list of gradients and the list of
    their outputs (None: in place), and the device.  Refuses what the call does not take."""
    n = len(grads)
    read = _lists()
    if read is not None:
        items = (ctypes.c_int64 * (4 * n))()               # GradItem is four 64-bit words
        index = read(grads, outs, _DL_CUDA, ctypes.addressof(items))
        if index >= 0:
            return items, ctypes.addressof(items), torch.device("cuda", index)
    # refused, or tensors of a class of their own: by their attributes, whole lists at a time
    dev, index = grads[0].device, grads[0].get_device()
    kinds, sizes = [g.dtype for g in grads], [g.numel() for g in grads]
    if (index < 0 or not _DTYPES.keys() >= set(kinds) or [g.get_device() for g in grads].count(index) != n
            or False in [g.is_contiguous() for g in grads]):
        raise ValueError("gradients must be contiguous bfloat16 or float32 tensors on one CUDA device")
    if outs is not None and ([o.dtype for o in outs] != kinds or [o.numel() for o in outs] != sizes
                             or [o.get_device() for o in outs].count(index) != n
                             or False in [o.is_contiguous() for o in outs]):
        raise ValueError("out tensors must be contiguous and of their gradients' type, size and device")
    words = [0] * (4 * n)
    words[0::4] = [g.data_ptr() for g in grads]
    words[1::4] = words[0::4] if outs is None else [o.data_ptr() for o in outs]
    words[2::4], words[3::4] = sizes, [_DTYPES[k] for k in kinds]
    items = array.array("q", words)
    return items, items.buffer_info()[0], dev


def clip_grad_norm(grads, max_norm, eps=1e-6, out=None, stream=None):
    """Global L2 norm of a list of contiguous CUDA gradients (bfloat16 and float32, any shapes and sizes), and
    clipping by it: every gradient times min(1, max_norm / (norm + eps)), in place or into the tensors of the list
    `out` (same types and sizes; no overlap with other tensors).  Returns the norm before clipping as a float32
    CUDA tensor of shape () (nothing is read on the host)."""
    grads = list(grads)
    outs = None if out is None else list(out)
    if not grads:
        raise ValueError("no gradients")
    if outs is not None and len(outs) != len(grads):
        raise ValueError("out must have one tensor per gradient")
    n = len(grads)
    items, address, dev = _grad_items(grads, outs)
    nbytes = fp8q_clip_grad_workspace_bytes(n)
    with _on(dev, stream):
        ws = torch.empty(nbytes // 4 + 1, dtype=torch.float32, device=dev)     # the norm after the partial sums
        norm, base = ws[nbytes // 4], ws.data_ptr()
        st = fp8q_clip_grad_norm(ctypes.c_void_p(address), n, max_norm, eps,
                                 ctypes.c_void_p(base + nbytes), ctypes.c_void_p(base), nbytes, _stream())
    del items                                              # the call has read them
    _check(st, "fp8q_clip_grad_norm")
    _results(stream, norm)
    return norm


def device_status(stream=None):
    """Synchronizes the stream; returns and clears the device status word."""
    return fp8q_get_device_status(_stream(stream))
