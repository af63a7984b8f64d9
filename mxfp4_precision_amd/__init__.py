"""Python binding of libmxfp4 (MXFP4 quantize + block-scaled a4w4 GEMM for gfx950).

Argument marshalling only: every step of the path runs in the HIP kernels of
``libmxfp4.so``.  Functions carry the C ABI's names (``include/mxfp4.h``) and
take device pointers as ints or GPU torch tensors (their ``data_ptr()``; host
tensors and arrays are refused before any call), sizes as ints, and a stream
as a ``torch.cuda.Stream``, an int handle, or None (torch's current stream).
A non-zero status raises ``MXError``; if the shared library is missing, the
first call raises: there is no fallback.

Build the library with ``python -m mxfp4_precision_amd.build``.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Tuple

_HERE = os.path.dirname(os.path.abspath(__file__))
# MXFP4_LIB names another build of the same library (the sanitizer build of
# the host code that the CPU tests run); the default is the in-tree build.
LIB_PATH = os.environ.get("MXFP4_LIB") or os.path.join(_HERE, "libmxfp4.so")

MX_SUCCESS = 0
MX_ERR_INVALID_ARGUMENT = 1
MX_ERR_MISALIGNED = 2
MX_ERR_UNSUPPORTED = 3
MX_ERR_DEVICE_UNSUPPORTED = 4
MX_ERR_HIP = 5

MX_LAYOUT_CANONICAL = 0
MX_LAYOUT_TILED = 1
MX_BF16 = 0
MX_F32 = 1
MX_FP6_E2M3 = 2
MX_FP6_E3M2 = 3
MX_STATE_F32 = 0
MX_STATE_MXFP8 = 1

EXPORTED = ("mx_blob_bytes", "mx_quantize_rowwise", "mx_quantize_dual", "mx_gemm_a4w4", "mx_gemm_a4w4_bias",
            "mx_layout_convert", "mx_layout_convert_host", "mx_dequantize", "mx_device_supported",
            "mx_fp8_blob_bytes", "mx_quantize_fp8_tw", "mx_gemm_f8_tw",
            "mx_fp6_blob_bytes", "mx_quantize_fp6", "mx_gemm_fp6", "mx_quantize_dual_mul",
            "mx_grouped_blob_bytes", "mx_quantize_grouped", "mx_gemm_a4w4_grouped", "mx_gemm_a4w4_grouped_wgrad",
            "mx_adamw", "mx_adamw_step_values",
            "mx_measure_mfma", "mx_set_device_arch_override", "mx_status_string", "mx_last_error")


class MXError(RuntimeError):
    def __init__(self, status: int, detail: str):
        super().__init__("%s: %s" % (_status_name(status), detail))
        self.status = status


class mx_quant_opts(ctypes.Structure):
    _fields_ = [("use_2d_block", ctypes.c_uint32), ("use_sr", ctypes.c_uint32),
                ("seed", ctypes.c_uint64), ("tensor_id", ctypes.c_uint32),
                ("index_base", ctypes.c_uint64), ("rht", ctypes.c_uint32)]


def quant_opts(use_2d_block: bool = False, use_sr: bool = False, seed: int = 0,
               tensor_id: int = 0, index_base: int = 0, rht: int = 0) -> mx_quant_opts:
    return mx_quant_opts(int(use_2d_block), int(use_sr), seed, tensor_id, index_base, rht)


class mx_adamw_step(ctypes.Structure):
    _fields_ = [("grad_scale", ctypes.c_float), ("decay", ctypes.c_float), ("step_size", ctypes.c_float),
                ("root_factor", ctypes.c_float), ("seed", ctypes.c_uint64)]


class mx_adamw_tensor(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("grad", ctypes.c_void_p), ("exp_avg", ctypes.c_void_p),
                ("exp_avg_sq", ctypes.c_void_p), ("exp_avg_scale", ctypes.c_void_p),
                ("exp_avg_sq_scale", ctypes.c_void_p), ("param_copy", ctypes.c_void_p), ("numel", ctypes.c_int64),
                ("tensor_id", ctypes.c_uint32)]


class mx_adamw_opts(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("weight_decay", ctypes.c_double), ("step", ctypes.c_int64),
                ("grad_scale", ctypes.c_double), ("seed", ctypes.c_uint64), ("param_dtype", ctypes.c_int),
                ("grad_dtype", ctypes.c_int), ("state_dtype", ctypes.c_int), ("use_sr", ctypes.c_uint32),
                ("device_step", ctypes.c_void_p)]


def adamw_opts(lr: float, step: int, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
               weight_decay: float = 0.0, grad_scale: float = 1.0, seed: int = 0, param_dtype: int = MX_F32,
               grad_dtype: int = MX_BF16, state_dtype: int = MX_STATE_F32, use_sr: bool = False,
               device_step=None) -> mx_adamw_opts:
    """device_step: a GPU tensor that holds an mx_adamw_step (24 bytes); the caller keeps it alive."""
    return mx_adamw_opts(lr, beta1, beta2, eps, weight_decay, step, grad_scale, seed, param_dtype, grad_dtype,
                         state_dtype, int(use_sr), _dptr(device_step))


def adamw_tensor(param, grad, exp_avg, exp_avg_sq, numel: int, exp_avg_scale=None, exp_avg_sq_scale=None,
                 param_copy=None, tensor_id: int = 0) -> mx_adamw_tensor:
    """One row of an mx_adamw table.  It holds addresses: the caller keeps the tensors alive."""
    return mx_adamw_tensor(_dptr(param), _dptr(grad), _dptr(exp_avg), _dptr(exp_avg_sq), _dptr(exp_avg_scale),
                           _dptr(exp_avg_sq_scale), _dptr(param_copy), numel, tensor_id)


def adamw_table(rows):
    """The host array of mx_adamw (built once, used every step while the addresses stay)."""
    return (mx_adamw_tensor * max(len(rows), 1))(*rows)


try:
    from . import _marshal      # converts the arguments of the grouped calls (csrc/marshal.cpp)
except ImportError:
    _marshal = None             # the same conversions in Python

_lib = None


def lib() -> ctypes.CDLL:
    """Load libmxfp4.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError("libmxfp4.so not found at %s: build it with "
                           "`python -m mxfp4_precision_amd.build` (no fallback path exists)" % LIB_PATH)
    L = ctypes.CDLL(LIB_PATH)
    i64, vp, i32 = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int
    optp = ctypes.POINTER(mx_quant_opts)
    L.mx_blob_bytes.argtypes = [i64, i64, i32, ctypes.POINTER(ctypes.c_size_t), ctypes.POINTER(ctypes.c_size_t)]
    L.mx_quantize_rowwise.argtypes = [vp, i64, i64, i64, optp, i32, vp, vp, vp]
    L.mx_quantize_dual.argtypes = [vp, i64, i64, i64, optp, optp, i32, vp, vp, vp, vp, vp]
    L.mx_gemm_a4w4.argtypes = [i32, i32, i64, i64, i64, vp, vp, vp, vp, i32, i32, vp, i64, vp]
    L.mx_gemm_a4w4_bias.argtypes = [i32, i32, i64, i64, i64, vp, vp, vp, vp, i32, i32, vp, vp, i64, vp]
    L.mx_layout_convert.argtypes = [i32, i64, i64, vp, vp, vp, vp, vp]
    L.mx_fp8_blob_bytes.argtypes = [i64, i64, i32, ctypes.POINTER(ctypes.c_size_t)]
    L.mx_quantize_fp8_tw.argtypes = [vp, i64, i64, i64, i32, vp, vp, vp, vp]
    L.mx_gemm_f8_tw.argtypes = [i32, i32, i64, i64, i64, vp, vp, vp, vp, i32, i32, vp, i64, vp]
    L.mx_layout_convert_host.argtypes = [i32, i64, i64, vp, vp, vp, vp]
    L.mx_fp6_blob_bytes.argtypes = [i64, i64, i32, ctypes.POINTER(ctypes.c_size_t), ctypes.POINTER(ctypes.c_size_t)]
    L.mx_quantize_fp6.argtypes = [vp, i64, i64, i64, i32, optp, i32, optp, i32, vp, vp, vp, vp, vp]
    L.mx_quantize_dual_mul.argtypes = [vp, vp, i64, i64, i64, i64, optp, optp, i32, vp, vp, vp, vp, vp]
    L.mx_gemm_fp6.argtypes = [i32, i32, i64, i64, i64, i32, vp, vp, i32, vp, vp, i32, i32, vp, i64, vp]
    szp = ctypes.POINTER(ctypes.c_size_t)
    L.mx_grouped_blob_bytes.argtypes = [i64, i64, i32, szp, szp, szp, szp]
    L.mx_quantize_grouped.argtypes = [vp, i64, i64, i64, vp, i64, vp, i32, optp, optp, i32, vp, vp, vp, vp, vp]
    L.mx_gemm_a4w4_grouped.argtypes = [i64, i64, i64, vp, i32, vp, vp, vp, vp, i32, i32, vp, vp, i64, vp]
    L.mx_gemm_a4w4_grouped_wgrad.argtypes = [i64, i64, i64, vp, i32, vp, vp, vp, vp, i32, i32, vp, i64, i64, vp]
    L.mx_adamw.argtypes = [ctypes.POINTER(mx_adamw_tensor), i64, ctypes.POINTER(mx_adamw_opts), vp]
    L.mx_adamw_step_values.argtypes = [ctypes.POINTER(mx_adamw_opts), ctypes.POINTER(mx_adamw_step)]
    L.mx_dequantize.argtypes = [vp, vp, i64, i64, i32, vp, i64, vp]
    L.mx_measure_mfma.argtypes = [i32, i32, vp, i32, i64, vp, vp]
    L.mx_set_device_arch_override.argtypes = [ctypes.c_char_p]
    L.mx_device_supported.argtypes = [i32]
    L.mx_device_supported.restype = i32
    L.mx_status_string.argtypes = [i32]
    L.mx_status_string.restype = ctypes.c_char_p
    L.mx_last_error.argtypes = []
    L.mx_last_error.restype = ctypes.c_char_p
    for name in EXPORTED:
        if name not in ("mx_device_supported", "mx_status_string", "mx_last_error"):
            getattr(L, name).restype = i32     # mx_status
    if _marshal is not None:
        address = lambda f: ctypes.cast(f, vp).value  # noqa: E731
        _marshal.bind(address(L.mx_quantize_grouped), address(L.mx_gemm_a4w4_grouped),
                      address(L.mx_gemm_a4w4_grouped_wgrad), _dptr, _i32ptr, _stream, mx_quant_opts)
    _lib = L
    return L


def _status_name(st: int) -> str:
    try:
        return lib().mx_status_string(st).decode()
    except Exception:
        return "status %d" % st


def _check(st: int):
    if st != MX_SUCCESS:
        raise MXError(st, lib().mx_last_error().decode())


def _dptr(p) -> Optional[int]:
    """A device-pointer argument.  Ints pass through (the caller vouches for
    them); a tensor must live on a GPU.  Host tensors and arrays are refused
    here: a kernel that dereferences a host address faults the device."""
    if p is None or isinstance(p, int):
        return p
    if getattr(p, "is_cuda", False):
        return p.data_ptr()
    if hasattr(p, "data_ptr"):
        raise TypeError("a device pointer is required, got a tensor on %s" % p.device)
    raise TypeError("a device pointer is required, got %r (host arrays are not accepted)" % type(p))


def _i32ptr(p, count: int) -> Optional[int]:
    """A device pointer to `count` int32 values.  A tensor of another type, with gaps or with fewer values is
    refused: the kernels read that many consecutive 32-bit words."""
    if p is not None and not isinstance(p, int) and hasattr(p, "data_ptr"):
        if str(p.dtype) != "torch.int32" or not p.is_contiguous() or p.numel() < count:
            raise TypeError("a contiguous int32 tensor of at least %d values is required, got %s of %s"
                            % (count, p.dtype, tuple(p.shape)))
    return _dptr(p)


def _hptr(p) -> Optional[int]:
    """A host-pointer argument (the host layout converter): numpy arrays, CPU
    tensors or ints; device tensors are refused."""
    if p is None or isinstance(p, int):
        return p
    if hasattr(p, "data_ptr"):
        if getattr(p, "is_cuda", False):
            raise TypeError("a host pointer is required, got a tensor on %s" % p.device)
        return p.data_ptr()
    if hasattr(p, "ctypes"):          # numpy array
        return p.ctypes.data
    raise TypeError("expected a host array, tensor or int, got %r" % type(p))


def _current_stream() -> int:
    """The handle of torch's current stream.  torch.cuda.current_stream() builds a Stream object for it, which took
    2.7 us of a 7.7 us call; the handle alone takes 0.2 us."""
    global _current_stream
    import torch
    device, raw = getattr(torch._C, "_cuda_getDevice", None), getattr(torch._C, "_cuda_getCurrentRawStream", None)
    torch.cuda.current_stream()     # initializes torch's CUDA state, which the two functions expect
    if device and raw:
        _current_stream = lambda: raw(device())  # noqa: E731
    else:
        _current_stream = lambda: torch.cuda.current_stream().cuda_stream  # noqa: E731
    return _current_stream()


def _stream(s) -> Optional[int]:
    if s is None:
        return _current_stream()
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _opts(o):
    return ctypes.byref(o) if o is not None else None


# ------------------------------------------------------------------ C ABI names

def mx_blob_bytes(rows: int, length: int, layout: int) -> Tuple[int, int]:
    d, s = ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib().mx_blob_bytes(rows, length, layout, ctypes.byref(d), ctypes.byref(s)))
    return d.value, s.value


def mx_quantize_rowwise(x, M: int, N: int, ldx: int, opts, layout: int, q, s, stream=None):
    _check(lib().mx_quantize_rowwise(_dptr(x), M, N, ldx, _opts(opts), layout, _dptr(q), _dptr(s),
                                     _stream(stream)))


def mx_quantize_dual(x, M: int, N: int, ldx: int, row_opts, col_opts, layout: int,
                     q_row, s_row, q_col, s_col, stream=None):
    _check(lib().mx_quantize_dual(_dptr(x), M, N, ldx, _opts(row_opts), _opts(col_opts), layout,
                                  _dptr(q_row), _dptr(s_row), _dptr(q_col), _dptr(s_col), _stream(stream)))


def mx_quantize_dual_mul(x, g, M: int, N: int, ldx: int, ldg: int, row_opts, col_opts, layout: int,
                         q_row, s_row, q_col=None, s_col=None, stream=None):
    _check(lib().mx_quantize_dual_mul(_dptr(x), _dptr(g), M, N, ldx, ldg, _opts(row_opts), _opts(col_opts),
                                      layout, _dptr(q_row), _dptr(s_row), _dptr(q_col), _dptr(s_col),
                                      _stream(stream)))


def mx_fp6_blob_bytes(rows: int, length: int, layout: int) -> Tuple[int, int]:
    d, s = ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib().mx_fp6_blob_bytes(rows, length, layout, ctypes.byref(d), ctypes.byref(s)))
    return d.value, s.value


def mx_quantize_fp6(x, M: int, N: int, ldx: int, row_fmt: int, row_opts, col_fmt: int, col_opts,
                    layout: int, q_row, s_row, q_col=None, s_col=None, stream=None):
    _check(lib().mx_quantize_fp6(_dptr(x), M, N, ldx, row_fmt, _opts(row_opts), col_fmt, _opts(col_opts),
                                 layout, _dptr(q_row), _dptr(s_row), _dptr(q_col), _dptr(s_col), _stream(stream)))


def mx_gemm_fp6(transA: int, transB: int, M: int, N: int, K: int, fmt_a: int, A, A_scale, fmt_b: int, B, B_scale,
                layout: int, out_dtype: int, C, ldc: int, stream=None):
    _check(lib().mx_gemm_fp6(transA, transB, M, N, K, fmt_a, _dptr(A), _dptr(A_scale), fmt_b, _dptr(B),
                             _dptr(B_scale), layout, out_dtype, _dptr(C), ldc, _stream(stream)))


def mx_gemm_a4w4(transA: int, transB: int, M: int, N: int, K: int, A, A_scale, B, B_scale,
                 layout: int, out_dtype: int, C, ldc: int, stream=None):
    _check(lib().mx_gemm_a4w4(transA, transB, M, N, K, _dptr(A), _dptr(A_scale), _dptr(B), _dptr(B_scale),
                              layout, out_dtype, _dptr(C), ldc, _stream(stream)))


def mx_gemm_a4w4_bias(transA: int, transB: int, M: int, N: int, K: int, A, A_scale, B, B_scale,
                      layout: int, out_dtype: int, bias, C, ldc: int, stream=None):
    _check(lib().mx_gemm_a4w4_bias(transA, transB, M, N, K, _dptr(A), _dptr(A_scale), _dptr(B), _dptr(B_scale),
                                   layout, out_dtype, _dptr(bias), _dptr(C), ldc, _stream(stream)))


def mx_fp8_blob_bytes(rows: int, length: int, layout: int) -> int:
    n = ctypes.c_size_t()
    _check(lib().mx_fp8_blob_bytes(rows, length, layout, ctypes.byref(n)))
    return n.value


def mx_quantize_fp8_tw(x, M: int, N: int, ldx: int, layout: int, q_row, q_col, info, stream=None):
    _check(lib().mx_quantize_fp8_tw(_dptr(x), M, N, ldx, layout, _dptr(q_row), _dptr(q_col), _dptr(info),
                                    _stream(stream)))


def mx_gemm_f8_tw(transA: int, transB: int, M: int, N: int, K: int, A, a_scale_inv, B, b_scale_inv,
                  layout: int, out_dtype: int, C, ldc: int, stream=None):
    _check(lib().mx_gemm_f8_tw(transA, transB, M, N, K, _dptr(A), _dptr(a_scale_inv), _dptr(B),
                               _dptr(b_scale_inv), layout, out_dtype, _dptr(C), ldc, _stream(stream)))


def mx_grouped_blob_bytes(M: int, N: int, groups: int) -> Tuple[int, int, int, int]:
    """(row data, row scales, column data, column scales): the most bytes that M rows in `groups` groups need."""
    n = [ctypes.c_size_t() for _ in range(4)]
    _check(lib().mx_grouped_blob_bytes(M, N, groups, *(ctypes.byref(v) for v in n)))
    return tuple(v.value for v in n)


def mx_quantize_grouped(x, x_rows: int, N: int, ldx: int, row_index, M: int, group_ends, groups: int, row_opts,
                        col_opts, layout: int, q_row, s_row, q_col=None, s_col=None, stream=None):
    L = lib()
    if _marshal is not None:
        _check(_marshal.quantize_grouped(x, x_rows, N, ldx, row_index, M, group_ends, groups, row_opts, col_opts,
                                         layout, q_row, s_row, q_col, s_col, stream))
        return
    _check(L.mx_quantize_grouped(_dptr(x), x_rows, N, ldx, _i32ptr(row_index, M), M, _i32ptr(group_ends, groups),
                                 groups, _opts(row_opts), _opts(col_opts), layout, _dptr(q_row), _dptr(s_row),
                                 _dptr(q_col), _dptr(s_col), _stream(stream)))


def mx_gemm_a4w4_grouped(M: int, N: int, K: int, group_ends, groups: int, A, A_scale, B, B_scale, layout: int,
                         out_dtype: int, bias, C, ldc: int, stream=None):
    L = lib()
    if _marshal is not None:
        _check(_marshal.gemm_grouped(M, N, K, group_ends, groups, A, A_scale, B, B_scale, layout, out_dtype, bias, C,
                                     ldc, stream))
        return
    _check(L.mx_gemm_a4w4_grouped(M, N, K, _i32ptr(group_ends, groups), groups, _dptr(A), _dptr(A_scale), _dptr(B),
                                  _dptr(B_scale), layout, out_dtype, _dptr(bias), _dptr(C), ldc, _stream(stream)))


def mx_gemm_a4w4_grouped_wgrad(M: int, N: int, K: int, group_ends, groups: int, A, A_scale, B, B_scale, layout: int,
                               out_dtype: int, C, ldc: int, group_stride: int, stream=None):
    L = lib()
    if _marshal is not None:
        _check(_marshal.gemm_grouped_wgrad(M, N, K, group_ends, groups, A, A_scale, B, B_scale, layout, out_dtype, C,
                                           ldc, group_stride, stream))
        return
    _check(L.mx_gemm_a4w4_grouped_wgrad(M, N, K, _i32ptr(group_ends, groups), groups, _dptr(A), _dptr(A_scale),
                                        _dptr(B), _dptr(B_scale), layout, out_dtype, _dptr(C), ldc, group_stride,
                                        _stream(stream)))


def mx_adamw(tensors, count: int, opts: mx_adamw_opts, stream=None):
    """tensors: an array of adamw_table.  count may not exceed its length."""
    if tensors is not None and count > len(tensors):
        raise ValueError("count=%d, but the table holds %d tensors" % (count, len(tensors)))
    _check(lib().mx_adamw(tensors, count, ctypes.byref(opts), _stream(stream)))


def mx_adamw_step_values(opts: mx_adamw_opts) -> mx_adamw_step:
    step = mx_adamw_step()
    _check(lib().mx_adamw_step_values(ctypes.byref(opts), ctypes.byref(step)))
    return step


def mx_layout_convert(to_tiled: int, rows: int, length: int, q_src, s_src, q_dst, s_dst, stream=None):
    _check(lib().mx_layout_convert(to_tiled, rows, length, _dptr(q_src), _dptr(s_src), _dptr(q_dst),
                                   _dptr(s_dst), _stream(stream)))


def mx_layout_convert_host(to_tiled: int, rows: int, length: int, q_src, s_src, q_dst, s_dst):
    _check(lib().mx_layout_convert_host(to_tiled, rows, length, _hptr(q_src), _hptr(s_src),
                                        _hptr(q_dst), _hptr(s_dst)))


def mx_dequantize(q, s, rows: int, length: int, layout: int, out_f32, ldo: int, stream=None):
    _check(lib().mx_dequantize(_dptr(q), _dptr(s), rows, length, layout, _dptr(out_f32), ldo,
                               _stream(stream)))


def mx_measure_mfma(fmt_a: int, fmt_b: int, operands, workgroups: int, iters: int, out, stream=None):
    _check(lib().mx_measure_mfma(fmt_a, fmt_b, _dptr(operands), workgroups, iters, _dptr(out), _stream(stream)))


def mx_device_supported(device: int) -> bool:
    return bool(lib().mx_device_supported(device))


def mx_set_device_arch_override(arch: Optional[str]):
    """Test aid: fixed architecture name in place of the device query (None restores it)."""
    _check(lib().mx_set_device_arch_override(None if arch is None else arch.encode()))


def mx_status_string(status: int) -> str:
    return lib().mx_status_string(status).decode()


def mx_last_error() -> str:
    return lib().mx_last_error().decode()


# ------------------------------------------------- allocation helpers (plumbing)

def empty_blob(rows: int, length: int, layout: int, device="cuda"):
    """Allocate (data, scale) uint8 tensors of the right byte sizes on `device`."""
    import torch
    db, sb = mx_blob_bytes(rows, length, layout)
    return (torch.empty(max(db, 1), dtype=torch.uint8, device=device),
            torch.empty(max(sb, 1), dtype=torch.uint8, device=device))


def empty_grouped_blob(M: int, N: int, groups: int, device="cuda"):
    """Allocate (row data, row scales, column data, column scales) uint8 tensors for any split of M rows of N
    elements into `groups` groups."""
    import torch
    return tuple(torch.empty(max(n, 1), dtype=torch.uint8, device=device) for n in mx_grouped_blob_bytes(M, N, groups))
