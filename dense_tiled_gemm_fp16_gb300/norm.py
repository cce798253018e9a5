"""The root-mean-square norm on CUDA torch tensors.

Mirrors ``include/rms_norm.h`` (as ``rms_norm_ptr``) and adds the tensor form
``rms_norm``, whose output can be the ``Fp8Matrix`` that the 8-bit products take.
"""
from __future__ import annotations

import ctypes

from .fp8 import BF16, Fp8Matrix, _cuda, _dtype_code
from .mxf4 import _empty, _pkg, _run, _stream, _torch

MAX_DIM = 32768

# Every symbol include/rms_norm.h declares.
EXPORTED = ("rms_norm",)


def declare(L) -> None:
    """Argument types of the header's function on the loaded library."""
    P, I64, I = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    L.rms_norm.argtypes = [P, I, I64, P, I64, P, ctypes.c_float, P, I64, P, I64, P, P, I64, I64, P]
    L.rms_norm.restype = I


def rms_norm_ptr(x: int, dtype: int, stride_x: int, residual: int, stride_residual: int, weight: int, eps: float,
                 sum: int, stride_sum: int, y: int, stride_y: int, codes: int, scales: int, rows: int, d: int,
                 stream: int = 0) -> None:
    """rms_norm on device pointers, 0 for what is absent (see include/rms_norm.h)."""
    g = _pkg()
    g._check(g.lib().rms_norm(x, dtype, stride_x, residual or None, stride_residual, weight, eps, sum or None,
                              stride_sum, y or None, stride_y, codes or None, scales or None, rows, d, stream or None),
             "rms_norm")


def _rows(v, shape, dtype, device, name: str) -> int:
    """The row stride of v, a matrix of that shape, type and device with contiguous rows."""
    if v.shape != shape or v.dtype is not dtype:
        raise ValueError(f"{name} must have x's shape and type")
    if v.device != device:
        raise ValueError("tensors must share one CUDA device")
    s, unit = v.stride()
    if unit != 1 and shape[1] > 1:
        raise ValueError(f"{name} must have contiguous rows")
    return s if shape[0] > 1 else max(shape[1], 1)


def rms_norm(x, weight, eps: float = 1e-6, residual=None, quantize: bool = False, out=None, sum_out=None, stream=None):
    """h / sqrt(mean(h^2) + eps) * weight for the rows h of x [rows, d], or of x +
    residual: float16 or bfloat16, rows contiguous, weight [d] of the same type.

    Returns y [rows, d] of x's type, or with `quantize` the Fp8Matrix of it, and
    with a residual (y, h), h the sum rounded to x's type; `sum_out` receives h and
    may be x or residual itself."""
    shape, dtype, device = x.shape, x.dtype, x.device
    if len(shape) != 2:
        raise ValueError("rms_norm takes x [rows, d]")
    code = _dtype_code(dtype, "x", BF16)
    rows, d = shape
    sx, unit = x.stride()
    if unit != 1 and d > 1:
        raise ValueError("x must have contiguous rows")
    if rows < 2:
        sx = max(d, 1)
    if weight.shape != shape[1:] or weight.dtype is not dtype or (d > 1 and weight.stride(0) != 1):
        raise ValueError("weight must hold d values of x's type with unit stride")
    if weight.device != device:
        raise ValueError("tensors must share one CUDA device")
    _cuda(device)
    h, hp, rp, sr, ss, sy = None, None, None, 0, d, d
    if residual is not None:
        sr = _rows(residual, shape, dtype, device, "residual")
        if sum_out is None:
            h = _empty(shape, dtype, device, stream)
        else:
            h, ss = sum_out, _rows(sum_out, shape, dtype, device, "sum_out")
        hp, rp = h.data_ptr(), residual.data_ptr()
    elif sum_out is not None:
        raise ValueError("sum_out needs a residual")
    yp = cp = sp = None
    if quantize:
        if out is not None:
            raise ValueError("out is for an output that is not quantized")
        if rows < 1 or d < 1:
            raise ValueError("a matrix in 8 bits has at least one row and one value")
        y = Fp8Matrix._new(rows, d, None, device, stream)
        cp, sp = y.codes_ptr, y.scales_ptr
    else:
        if out is None:
            y = _empty(shape, dtype, device, stream)
        else:
            y, sy = out, _rows(out, shape, dtype, device, "out")
        yp = y.data_ptr()
    if rows:
        _run(device, "rms_norm", x.data_ptr(), code, sx, rp, sr, weight.data_ptr(), eps, hp, ss, yp, sy, cp, sp, rows, d,
             _stream(device, stream))
    return y if residual is None else (y, h)
