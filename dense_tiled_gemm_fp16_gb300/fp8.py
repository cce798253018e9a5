"""8-bit matrices on CUDA torch tensors: quantisation, its inverse, the product and the grouped product.

Mirrors ``include/gemm_fp8.h`` (``fp8_sizes``, ``gemm_fp8``, ``gemm_fp8_a16``,
``gemm_fp8_grouped``, ``gemm_fp8_grouped_a16`` and the pointer forms of the two
conversions) and adds the tensor forms ``fp8_quantize``, ``fp8_dequantize``,
``fp8_mm`` and ``fp8_grouped_mm``.  Like the rest of the binding it only marshals
arguments; PyTorch supplies memory and streams.
"""
from __future__ import annotations

import ctypes

from .mxf4 import BF16, F16, F32, _empty, _pkg, _run, _stream, _torch  # noqa: F401

MAX_GROUPS = 512

# Every symbol include/gemm_fp8.h declares.
EXPORTED = ("fp8_sizes", "fp8_quantize", "fp8_dequantize", "gemm_fp8", "gemm_fp8_a16", "gemm_fp8_grouped",
            "gemm_fp8_grouped_a16")


def declare(L) -> None:
    """Argument types of the header's functions on the loaded library."""
    P, I64, I = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    L.fp8_sizes.argtypes = [I64, I64, I64, ctypes.POINTER(I64), ctypes.POINTER(I64)]
    L.fp8_quantize.argtypes = [P, I, I64, I64, I64, P, P, I64, I64, I64, P]
    L.fp8_dequantize.argtypes = [P, P, P, I, I64, I64, I64, P]
    L.gemm_fp8.argtypes = [P, P, P, P, P, I, P, I, I64, I64, I64, I64, P]
    L.gemm_fp8_a16.argtypes = [P, I, I64, I64, P, P, P, P, I, P, I, I64, I64, I64, I64, P]
    L.gemm_fp8_grouped.argtypes = [P, P, P, P, P, P, P, I, P, I, I64, I64, I64, I64, I64, P]
    L.gemm_fp8_grouped_a16.argtypes = [P, I, I64, I64, P, P, P, P, P, P, I, P, I, I64, I64, I64, I64, I64, P]
    for name in EXPORTED:
        getattr(L, name).restype = I


# ------------------------------------------------------------ C-ABI mirrors
def fp8_sizes(rows: int, k: int, batch: int = 1):
    """(bytes of the codes, bytes of the scales) of `batch` matrices."""
    g = _pkg()
    c, s = ctypes.c_int64(0), ctypes.c_int64(0)
    g._check(g.lib().fp8_sizes(rows, k, batch, ctypes.byref(c), ctypes.byref(s)), "fp8_sizes")
    return c.value, s.value


def fp8_quantize_ptr(x: int, dtype: int, stride_b: int, stride_r: int, stride_k: int, codes: int, scales: int,
                     rows: int, k: int, batch: int, stream: int = 0) -> None:
    """fp8_quantize on device pointers (see include/gemm_fp8.h)."""
    g = _pkg()
    g._check(g.lib().fp8_quantize(x, dtype, stride_b, stride_r, stride_k, codes, scales, rows, k, batch,
                                  stream or None), "fp8_quantize")


def fp8_dequantize_ptr(codes: int, scales: int, y: int, dtype: int, rows: int, k: int, batch: int,
                       stream: int = 0) -> None:
    """fp8_dequantize on device pointers (see include/gemm_fp8.h)."""
    g = _pkg()
    g._check(g.lib().fp8_dequantize(codes, scales, y, dtype, rows, k, batch, stream or None), "fp8_dequantize")


def gemm_fp8(A_codes: int, A_scales: int, B_codes: int, B_scales: int, bias: int, act: int, C: int, dtype: int,
             ldc: int, M: int, N: int, K: int, stream: int = 0) -> None:
    """C = act(A B^T + bias) on device pointers (see include/gemm_fp8.h)."""
    g = _pkg()
    g._check(g.lib().gemm_fp8(A_codes, A_scales, B_codes, B_scales, bias or None, act, C, dtype, ldc, M, N, K,
                              stream or None), "gemm_fp8")


def gemm_fp8_a16(A: int, a_dtype: int, stride_am: int, stride_ak: int, work: int, B_codes: int, B_scales: int,
                 bias: int, act: int, C: int, dtype: int, ldc: int, M: int, N: int, K: int, stream: int = 0) -> None:
    """gemm_fp8 with A in fp16 or bf16, quantised into `work` (see include/gemm_fp8.h)."""
    g = _pkg()
    g._check(g.lib().gemm_fp8_a16(A, a_dtype, stride_am, stride_ak, work, B_codes, B_scales, bias or None, act, C,
                                  dtype, ldc, M, N, K, stream or None), "gemm_fp8_a16")


def gemm_fp8_grouped(A_codes: int, A_scales: int, B_codes: int, B_scales: int, B_up_codes: int, B_up_scales: int,
                     group_rows: int, act: int, C: int, dtype: int, ldc: int, rows: int, groups: int, N: int, K: int,
                     stream: int = 0) -> None:
    """The grouped product on device pointers, group_rows among them (see include/gemm_fp8.h)."""
    g = _pkg()
    g._check(g.lib().gemm_fp8_grouped(A_codes, A_scales, B_codes, B_scales, B_up_codes or None, B_up_scales or None,
                                      group_rows, act, C, dtype, ldc, rows, groups, N, K, stream or None),
             "gemm_fp8_grouped")


def gemm_fp8_grouped_a16(A: int, a_dtype: int, stride_am: int, stride_ak: int, work: int, B_codes: int, B_scales: int,
                         B_up_codes: int, B_up_scales: int, group_rows: int, act: int, C: int, dtype: int, ldc: int,
                         rows: int, groups: int, N: int, K: int, stream: int = 0) -> None:
    """gemm_fp8_grouped with A in fp16 or bf16, quantised into `work` (see include/gemm_fp8.h)."""
    g = _pkg()
    g._check(g.lib().gemm_fp8_grouped_a16(A, a_dtype, stride_am, stride_ak, work, B_codes, B_scales,
                                          B_up_codes or None, B_up_scales or None, group_rows, act, C, dtype, ldc,
                                          rows, groups, N, K, stream or None), "gemm_fp8_grouped_a16")


# ------------------------------------------------------------ torch helpers
def _bytes(rows: int, k: int, batch: int):
    """fp8_sizes without its checks: (codes, scales)."""
    return batch * rows * ((k + 127) >> 7) * 128, batch * ((rows + 127) >> 7) * ((k + 511) >> 9) * 512


class Fp8Matrix:
    """A matrix [rows, k], or a batch [batch, rows, k], held in 8 bits along k:
    ``codes`` and ``scales`` are the byte arrays include/gemm_fp8.h lays out
    (contiguous uint8), ``codes_ptr`` and ``scales_ptr`` their device addresses."""

    __slots__ = ("_data", "_split", "rows", "k", "batch", "device", "codes_ptr", "scales_ptr")

    def __init__(self, codes, scales, rows: int, k: int, batch=None):
        u8 = _torch().uint8
        if codes.dtype is not u8 or scales.dtype is not u8:
            raise TypeError("codes and scales must be uint8 tensors")
        if min(rows, k, 1 if batch is None else batch) < 1:
            raise ValueError("a matrix has at least one row, one value and, in a batch, one matrix")
        if (codes.numel(), scales.numel()) != _bytes(rows, k, batch or 1) or codes.device != scales.device:
            raise ValueError("codes and scales do not hold a matrix of these sizes")
        if not codes.is_contiguous() or not scales.is_contiguous():   # (only their base addresses go on)
            raise ValueError("codes and scales must be contiguous")
        self._data, self._split = (codes, scales), None
        self.rows, self.k, self.batch, self.device = rows, k, batch, codes.device
        self.codes_ptr, self.scales_ptr = codes.data_ptr(), scales.data_ptr()

    @classmethod
    def _new(cls, rows: int, k: int, batch, device, stream):
        """An unwritten one, both arrays in one buffer, the scales first."""
        nc, ns = _bytes(rows, k, batch or 1)
        q = cls.__new__(cls)
        q._data, q._split = _empty(nc + ns, _torch().uint8, device, stream), ns
        q.rows, q.k, q.batch, q.device = rows, k, batch, device
        q.scales_ptr = p = q._data.data_ptr()
        q.codes_ptr = p + ns
        return q

    @property
    def codes(self):
        return self._data[0] if self._split is None else self._data[self._split:]

    @property
    def scales(self):
        return self._data[1] if self._split is None else self._data[:self._split]

    @property
    def shape(self):
        return (self.rows, self.k) if self.batch is None else (self.batch, self.rows, self.k)

    @property
    def nbytes(self) -> int:
        return sum(_bytes(self.rows, self.k, self.batch or 1))

    def __repr__(self):
        return f"Fp8Matrix{self.shape} on {self.device}"


_codes = {}   # torch dtype -> element type


def _dtype_code(dtype, what: str, most: int = F32) -> int:
    if not _codes:
        t = _torch()
        _codes.update({t.float16: F16, t.bfloat16: BF16, t.float32: F32})
    code = _codes.get(dtype)
    if code is None or code > most:
        raise TypeError(f"{what} must be float16{' or ' if most < F32 else ', '}bfloat16"
                        f"{'' if most < F32 else ' or float32'}")
    return code


def _cuda(device) -> None:
    if device.type != "cuda":
        raise ValueError("tensors must be on a CUDA device")


def fp8_quantize(x, axis: int = -1, stream=None) -> Fp8Matrix:
    """x (2-D, or 3-D with a leading batch; float16, bfloat16 or float32; any
    positive strides) in 8 bits along `axis`, the one a product will contract: a
    weight [K, N] takes axis=-2 and becomes the [N, K] matrix that fp8_mm and
    fp8_grouped_mm read."""
    shape, strides = x.shape, x.stride()
    nd = len(shape)
    if nd == 2:
        rows, k = shape
        sr, sk = strides
        held, batch, sb = None, 1, 0
    elif nd == 3:
        held, rows, k = shape
        sb, sr, sk = strides
        batch = held
        if batch == 1:
            sb = 0
    else:
        raise ValueError("fp8_quantize takes a matrix or a batch of matrices")
    if axis == -2 or axis == nd - 2:
        rows, k, sr, sk = k, rows, sk, sr
    elif axis != -1 and axis != nd - 1:
        raise ValueError("axis must be one of the two matrix dimensions")
    code = _dtype_code(x.dtype, "x")
    device = x.device
    _cuda(device)
    if min(rows, k, batch) < 1:
        raise ValueError("a matrix has at least one row, one value and, in a batch, one matrix")
    q = Fp8Matrix._new(rows, k, held, device, stream)
    # (a dimension of one element may carry any stride, a batch of stride 0 repeats)
    _run(device, "fp8_quantize", x.data_ptr(), code, sb, sr if rows > 1 else max(1, k), sk if k > 1 else 1, q.codes_ptr,
         q.scales_ptr, rows, k, batch, _stream(device, stream))
    return q


def fp8_dequantize(q: Fp8Matrix, dtype=None, stream=None):
    """The values of q, rounded once to `dtype` (float16 unless given)."""
    if not isinstance(q, Fp8Matrix):
        raise TypeError("fp8_dequantize takes an Fp8Matrix")
    if dtype is None:
        dtype = _torch().float16
    code = _dtype_code(dtype, "dtype")
    device = q.device
    _cuda(device)
    y = _empty(q.shape, dtype, device, stream)
    _run(device, "fp8_dequantize", q.codes_ptr, q.scales_ptr, y.data_ptr(), code, q.rows, q.k, q.batch or 1,
         _stream(device, stream))
    return y


def _output(shape, out, dtype, device, stream):
    """(out, its row pitch, its type's code): `out` checked, or a new [rows, N]."""
    if out is None:
        dtype = _torch().float16 if dtype is None else dtype
        code = _dtype_code(dtype, "dtype", BF16)
        return _empty(shape, dtype, device, stream), shape[1], code
    if dtype is not None and out.dtype is not dtype:
        raise TypeError("out must be of the given dtype")
    code = _dtype_code(out.dtype, "out", BF16)
    if out.device != device:
        raise ValueError("tensors must share one CUDA device")
    _pkg()._check_out(out, shape, "[rows, N]")
    return out, out.stride(0) if shape[0] > 1 else shape[1], code


def _left(a, b: Fp8Matrix, name: str):
    """(M, K) of the left operand, which is checked against b."""
    shape = a.shape
    if len(shape) != 2 or (not isinstance(a, Fp8Matrix) and a.dim() != 2):
        raise ValueError(f"{name} takes a as a matrix")
    if shape[1] != b.k:
        raise ValueError(f"inner dimensions differ: {shape[1]} vs {b.k}")
    if not isinstance(a, Fp8Matrix):
        _dtype_code(a.dtype, "a", BF16)
    _cuda(b.device)
    if a.device != b.device:
        raise ValueError("tensors must share one CUDA device")
    return shape[0], shape[1]


def fp8_mm(a, b: Fp8Matrix, bias=None, act="none", dtype=None, out=None, stream=None):
    """C[m, n] = act(sum_k a[m, k] b[n, k] + bias[n]) of type `dtype` (float16
    unless given, or bfloat16): b an Fp8Matrix [N, K], a an Fp8Matrix [M, K] or a
    float16 or bfloat16 tensor [M, K] that is quantised on the way; bias of C's
    type; returns C."""
    if not isinstance(b, Fp8Matrix) or b.batch is not None:
        raise TypeError("fp8_mm takes b as an Fp8Matrix of two dimensions")
    M, K = _left(a, b, "fp8_mm")
    N, device = b.rows, b.device
    act = _pkg()._act(act)
    out, ldc, code = _output((M, N), out, dtype, device, stream)
    bp = None
    if bias is not None:
        if bias.dim() != 1 or bias.shape[0] != N or (bias.stride(0) != 1 and N > 1):
            raise ValueError("bias must hold N values with unit stride")
        if bias.dtype is not out.dtype:
            raise TypeError("bias must be of the output's type")
        if bias.device != device:
            raise ValueError("tensors must share one CUDA device")
        bp = bias.data_ptr()
    s = _stream(device, stream)
    if isinstance(a, Fp8Matrix):
        _run(device, "gemm_fp8", a.codes_ptr, a.scales_ptr, b.codes_ptr, b.scales_ptr, bp, act, out.data_ptr(), code, ldc,
             M, N, K, s)
    else:
        sm, sk = a.stride()
        work = _empty(sum(_bytes(M, K, 1)), _torch().uint8, device, stream)
        _run(device, "gemm_fp8_a16", a.data_ptr(), _codes[a.dtype], sm if M > 1 else max(1, K), sk if K > 1 else 1,
             work.data_ptr(), b.codes_ptr, b.scales_ptr, bp, act, out.data_ptr(), code, ldc, M, N, K, s)
    return out


def fp8_grouped_mm(a, b: Fp8Matrix, group_rows, act="none", b_up=None, dtype=None, out=None, stream=None):
    """The grouped product: rows of `a` in consecutive groups, group g's times
    b[g], as act(a_g b[g]^T), or with b_up the gate/up form act(a_g b[g]^T) *
    (a_g b_up[g]^T).

    a is an Fp8Matrix [rows, K] or a float16 or bfloat16 tensor that is quantised
    on the way; b and b_up are Fp8Matrix batches [G, N, K] (``fp8_quantize(w,
    axis=-2)`` of weights [G, K, N]).  group_rows holds G int32 row counts on the
    same device, contiguous, and is read there: nothing waits for the host.  Rows
    past the groups' sum are left as they were in `out`.  Returns C [rows, N] of
    type `dtype` (float16 unless given, or bfloat16)."""
    if not isinstance(b, Fp8Matrix) or b.batch is None:
        raise TypeError("fp8_grouped_mm takes b as an Fp8Matrix batch")
    if b_up is not None and (not isinstance(b_up, Fp8Matrix) or b_up.shape != b.shape):
        raise TypeError("b_up must be an Fp8Matrix of b's shape")
    R, K = _left(a, b, "fp8_grouped_mm")
    N, G, device = b.rows, b.batch, b.device
    act = _pkg()._act(act)
    if group_rows.dtype is not _torch().int32 or group_rows.dim() != 1 or group_rows.shape[0] != G:
        raise TypeError("group_rows must be an int32 tensor with a count for each of b's matrices")
    if not group_rows.is_contiguous():
        raise ValueError("group_rows must be contiguous")
    if group_rows.device != device or (b_up is not None and b_up.device != device):
        raise ValueError("tensors must share one CUDA device")
    out, ldc, code = _output((R, N), out, dtype, device, stream)
    if R == 0:
        return out
    s = _stream(device, stream)
    up = (None, None) if b_up is None else (b_up.codes_ptr, b_up.scales_ptr)
    if isinstance(a, Fp8Matrix):
        _run(device, "gemm_fp8_grouped", a.codes_ptr, a.scales_ptr, b.codes_ptr, b.scales_ptr, *up, group_rows.data_ptr(),
             act, out.data_ptr(), code, ldc, R, G, N, K, s)
    else:
        sm, sk = a.stride()
        work = _empty(sum(_bytes(R, K, 1)), _torch().uint8, device, stream)
        _run(device, "gemm_fp8_grouped_a16", a.data_ptr(), _codes[a.dtype], sm if R > 1 else max(1, K), sk if K > 1 else 1,
             work.data_ptr(), b.codes_ptr, b.scales_ptr, *up, group_rows.data_ptr(), act, out.data_ptr(), code, ldc, R, G, N,
             K, s)
    return out
