"""Tokens in the order of their experts and back, on CUDA torch tensors.

Mirrors ``include/moe_route.h`` (its functions as ``.._ptr``) and adds the tensor
forms ``moe_sort``, ``moe_gather``, ``moe_combine`` and ``moe_combine_grad``: what
stands before and after a grouped product whose rows are (token, expert) choices.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

from .fp8 import BF16, Fp8Matrix, _cuda, _dtype_code
from .mxf4 import _empty, _pkg, _run, _stream, _torch

MAX_EXPERTS, MAX_TOP_K = 512, 32

# Every symbol include/moe_route.h declares.
EXPORTED = ("moe_sort_workspace_size", "moe_sort", "moe_gather", "moe_gather_fp8", "moe_combine", "moe_combine_grad")


def declare(L) -> None:
    """Argument types of the header's functions on the loaded library."""
    P, I64, I, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
    L.moe_sort_workspace_size.argtypes = [I64, I64, I64, ctypes.POINTER(SZ)]
    L.moe_sort.argtypes = [P, I64, I64, I64, P, P, P, P, SZ, P]
    L.moe_gather.argtypes = [P, I, I64, P, I64, I64, I64, P, I64, P]
    L.moe_gather_fp8.argtypes = [P, P, P, I64, I64, I64, P, P, P]
    L.moe_combine.argtypes = [P, I, I64, P, P, I64, I64, I64, P, I64, P]
    L.moe_combine_grad.argtypes = [P, I, I64, P, I64, P, P, I64, I64, I64, P, I64, P, P]
    for name in EXPORTED:
        getattr(L, name).restype = I


# ------------------------------------------------------------ C-ABI mirrors
def moe_sort_workspace_size(tokens: int, top_k: int, experts: int) -> int:
    g = _pkg()
    n = ctypes.c_size_t(0)
    g._check(g.lib().moe_sort_workspace_size(tokens, top_k, experts, ctypes.byref(n)), "moe_sort_workspace_size")
    return n.value


def moe_sort_ptr(ids: int, tokens: int, top_k: int, experts: int, rows: int, order: int, group_rows: int,
                 workspace: int, workspace_bytes: int, stream: int = 0) -> None:
    """moe_sort on device pointers (see include/moe_route.h)."""
    g = _pkg()
    g._check(g.lib().moe_sort(ids or None, tokens, top_k, experts, rows or None, order or None, group_rows or None,
                              workspace or None, workspace_bytes, stream or None), "moe_sort")


def moe_gather_ptr(x: int, dtype: int, stride_x: int, rows: int, tokens: int, top_k: int, d: int, out: int,
                   stride_out: int, stream: int = 0) -> None:
    """moe_gather on device pointers (see include/moe_route.h)."""
    g = _pkg()
    g._check(g.lib().moe_gather(x or None, dtype, stride_x, rows or None, tokens, top_k, d, out or None, stride_out,
                                stream or None), "moe_gather")


def moe_gather_fp8_ptr(codes: int, scales: int, rows: int, tokens: int, top_k: int, k: int, out_codes: int,
                       out_scales: int, stream: int = 0) -> None:
    """moe_gather_fp8 on device pointers (see include/moe_route.h)."""
    g = _pkg()
    g._check(g.lib().moe_gather_fp8(codes or None, scales or None, rows or None, tokens, top_k, k, out_codes or None,
                                    out_scales or None, stream or None), "moe_gather_fp8")


def moe_combine_ptr(y: int, dtype: int, stride_y: int, rows: int, weights: int, tokens: int, top_k: int, d: int,
                    out: int, stride_out: int, stream: int = 0) -> None:
    """moe_combine on device pointers (see include/moe_route.h)."""
    g = _pkg()
    g._check(g.lib().moe_combine(y or None, dtype, stride_y, rows or None, weights or None, tokens, top_k, d,
                                 out or None, stride_out, stream or None), "moe_combine")


def moe_combine_grad_ptr(dout: int, dtype: int, stride_dout: int, y: int, stride_y: int, rows: int, weights: int,
                         tokens: int, top_k: int, d: int, dy: int, stride_dy: int, dweights: int,
                         stream: int = 0) -> None:
    """moe_combine_grad on device pointers (see include/moe_route.h)."""
    g = _pkg()
    g._check(g.lib().moe_combine_grad(dout or None, dtype, stride_dout, y or None, stride_y, rows or None,
                                      weights or None, tokens, top_k, d, dy or None, stride_dy, dweights or None,
                                      stream or None), "moe_combine_grad")


# ------------------------------------------------------------ torch helpers
_FEW = 1024   # choices that moe_sort orders without a workspace


class MoeOrder(NamedTuple):
    """Where (token, expert) choices stand, int32 on the device: rows [T, top_k],
    the place of each choice (-1: no expert's); order [T * top_k], the choice t *
    top_k + j at each place (-1 past the last group); group_rows [experts], the
    choices of each expert, which fp8_grouped_mm takes."""
    rows: object
    order: object
    group_rows: object


def moe_sort(ids, experts: int, stream=None) -> MoeOrder:
    """The order of the choices ids [T, top_k] (int32, contiguous) by expert, of one
    expert by token.  An id outside 0 .. experts - 1 is no expert's."""
    t, shape, device = _torch(), ids.shape, ids.device
    if len(shape) != 2 or ids.dtype is not t.int32 or not ids.is_contiguous():
        raise TypeError("moe_sort takes ids as a contiguous int32 tensor [T, top_k]")
    T, top = shape
    n = T * top
    _cuda(device)
    need = moe_sort_workspace_size(T, top, experts) if n > _FEW or not 1 <= experts <= MAX_EXPERTS else 0
    rows, order, groups = (_empty(size, t.int32, device, stream) for size in (shape, n, experts))
    space = _empty(need, t.uint8, device, stream) if need else None
    _run(device, "moe_sort", ids.data_ptr() or None, T, top, experts, rows.data_ptr() or None, order.data_ptr() or None,
         groups.data_ptr(), space.data_ptr() if need else None, need, _stream(device, stream))
    return MoeOrder(rows, order, groups)


def _places(order: MoeOrder, device):
    """(T, top_k) of an order on `device`."""
    rows = order.rows
    shape = rows.shape
    if len(shape) != 2 or rows.dtype is not _torch().int32 or not rows.is_contiguous():
        raise TypeError("an order's rows are a contiguous int32 tensor [T, top_k]")
    if rows.device != device:
        raise ValueError("tensors must share one CUDA device")
    _cuda(device)
    return shape


def _matrix(v, shape, dtype, device, name: str) -> int:
    """The row stride of v, a matrix of that shape, type and device with contiguous rows."""
    if v.shape != shape or v.dtype is not dtype:
        raise ValueError(f"{name} must be {list(shape)} of type {dtype}")
    if v.device != device:
        raise ValueError("tensors must share one CUDA device")
    s, unit = v.stride()
    if unit != 1 and shape[1] > 1:
        raise ValueError(f"{name} must have contiguous rows")
    return s if shape[0] > 1 else max(1, shape[1])


def _weights(w, shape, device) -> None:
    if w.shape != shape or w.dtype is not _torch().float32 or not w.is_contiguous():
        raise TypeError("weights must be a contiguous float32 tensor [T, top_k]")
    if w.device != device:
        raise ValueError("tensors must share one CUDA device")


def moe_gather(x, order: MoeOrder, out=None, stream=None):
    """The rows of x [T, d] at the places of their tokens' choices, [T * top_k, d]:
    x float16 or bfloat16 with contiguous rows, or an Fp8Matrix (the result is one
    then, and `out` is not taken).  Places past the last group are left as they were.
    Its gradient is ``moe_combine(dout, order)``."""
    device = x.device
    T, top = _places(order, device)
    if len(x.shape) != 2 or x.shape[0] != T:
        raise ValueError("moe_gather takes x with a row for each token of the order")
    if isinstance(x, Fp8Matrix):
        if out is not None:
            raise ValueError("out is for a tensor x")
        q = Fp8Matrix._new(T * top, x.k, None, device, stream)
        _run(device, "moe_gather_fp8", x.codes_ptr, x.scales_ptr, order.rows.data_ptr(), T, top, x.k, q.codes_ptr,
             q.scales_ptr, _stream(device, stream))
        return q
    code, d = _dtype_code(x.dtype, "x", BF16), x.shape[1]
    sx = _matrix(x, (T, d), x.dtype, device, "x")
    so = d
    if out is None:
        out = _empty((T * top, d), x.dtype, device, stream)
    else:
        so = _matrix(out, (T * top, d), x.dtype, device, "out")
    if T:
        _run(device, "moe_gather", x.data_ptr(), code, sx, order.rows.data_ptr(), T, top, d, out.data_ptr(), so,
             _stream(device, stream))
    return out


def moe_combine(y, order: MoeOrder, weights=None, out=None, stream=None):
    """The rows of y [T * top_k, d] back by token: out[t] = sum_j weights[t, j]
    y[place of (t, j)] in fp32, rounded once, [T, d]; weights float32 [T, top_k], or
    None for ones.  Choices without a place add nothing."""
    device = y.device
    T, top = _places(order, device)
    if y.dim() != 2 or y.shape[0] != T * top:
        raise ValueError("moe_combine takes y with a row for each choice of the order")
    code, d = _dtype_code(y.dtype, "y", BF16), y.shape[1]
    sy = _matrix(y, (T * top, d), y.dtype, device, "y")
    if weights is not None:
        _weights(weights, (T, top), device)
    so = d
    if out is None:
        out = _empty((T, d), y.dtype, device, stream)
    else:
        so = _matrix(out, (T, d), y.dtype, device, "out")
    if T:
        _run(device, "moe_combine", y.data_ptr(), code, sy, order.rows.data_ptr(),
             None if weights is None else weights.data_ptr(), T, top, d, out.data_ptr(), so, _stream(device, stream))
    return out


def moe_combine_grad(dout, y, order: MoeOrder, weights, out=None, stream=None):
    """The gradient of moe_combine(y, order, weights) for dout [T, d]: (dy [T *
    top_k, d] of y's type, dweights [T, top_k] float32).  Rows of dy past the last
    group are left as they were; a choice without a place has a weight's gradient
    of 0."""
    device = y.device
    T, top = _places(order, device)
    if y.dim() != 2 or y.shape[0] != T * top:
        raise ValueError("moe_combine_grad takes y with a row for each choice of the order")
    code, d = _dtype_code(y.dtype, "y", BF16), y.shape[1]
    sy = _matrix(y, (T * top, d), y.dtype, device, "y")
    sg = _matrix(dout, (T, d), y.dtype, device, "dout")
    _weights(weights, (T, top), device)
    so = d
    if out is None:
        out = _empty((T * top, d), y.dtype, device, stream)
    else:
        so = _matrix(out, (T * top, d), y.dtype, device, "out")
    dw = _empty((T, top), weights.dtype, device, stream)
    if T:
        _run(device, "moe_combine_grad", dout.data_ptr(), code, sg, y.data_ptr(), sy, order.rows.data_ptr(),
             weights.data_ptr(), T, top, d, out.data_ptr(), so, dw.data_ptr(), _stream(device, stream))
    return out, dw
