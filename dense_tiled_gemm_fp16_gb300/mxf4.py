"""MXFP4 matrices on CUDA torch tensors: quantisation, its inverse and the product.

Mirrors ``include/gemm_mxf4.h`` (``mxf4_sizes``, ``gemm_mxf4`` and the pointer
forms of the two conversions) and adds the tensor forms ``mxf4_quantize``,
``mxf4_dequantize`` and ``mxf4_mm``.  Like the rest of the binding it only
marshals arguments; PyTorch supplies memory and streams.
"""
from __future__ import annotations

import ctypes

F16, BF16, F32 = range(3)

# Every symbol include/gemm_mxf4.h declares.
EXPORTED = ("mxf4_sizes", "mxf4_quantize", "mxf4_dequantize", "gemm_mxf4")


def declare(L) -> None:
    """Argument types of the header's functions on the loaded library."""
    P, I64, I = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    L.mxf4_sizes.argtypes = [I64, I64, I64, ctypes.POINTER(I64), ctypes.POINTER(I64)]
    L.mxf4_quantize.argtypes = [P, I, I64, I64, I64, P, P, I64, I64, I64, P]
    L.mxf4_dequantize.argtypes = [P, P, P, I, I64, I64, I64, P]
    L.gemm_mxf4.argtypes = [P, P, P, P, P, I, P, I64, I64, I64, I64, P]
    for name in EXPORTED:
        getattr(L, name).restype = I


def _pkg():
    import dense_tiled_gemm_fp16_gb300 as g
    return g


# ------------------------------------------------------------ C-ABI mirrors
def mxf4_sizes(rows: int, k: int, batch: int = 1):
    """(bytes of the codes, bytes of the scales) of `batch` matrices."""
    g = _pkg()
    c, s = ctypes.c_int64(0), ctypes.c_int64(0)
    g._check(g.lib().mxf4_sizes(rows, k, batch, ctypes.byref(c), ctypes.byref(s)), "mxf4_sizes")
    return c.value, s.value


def mxf4_quantize_ptr(x: int, dtype: int, stride_b: int, stride_r: int, stride_k: int, codes: int, scales: int,
                      rows: int, k: int, batch: int, stream: int = 0) -> None:
    """mxf4_quantize on device pointers (see include/gemm_mxf4.h)."""
    g = _pkg()
    g._check(g.lib().mxf4_quantize(x, dtype, stride_b, stride_r, stride_k, codes, scales, rows, k, batch,
                                   stream or None), "mxf4_quantize")


def mxf4_dequantize_ptr(codes: int, scales: int, y: int, dtype: int, rows: int, k: int, batch: int,
                        stream: int = 0) -> None:
    """mxf4_dequantize on device pointers (see include/gemm_mxf4.h)."""
    g = _pkg()
    g._check(g.lib().mxf4_dequantize(codes, scales, y, dtype, rows, k, batch, stream or None), "mxf4_dequantize")


def gemm_mxf4(A_codes: int, A_scales: int, B_codes: int, B_scales: int, bias: int, act: int, C: int, ldc: int, M: int,
              N: int, K: int, stream: int = 0) -> None:
    """C = act(A B^T + bias) on device pointers (see include/gemm_mxf4.h)."""
    g = _pkg()
    g._check(g.lib().gemm_mxf4(A_codes, A_scales, B_codes, B_scales, bias or None, act, C, ldc, M, N, K,
                               stream or None), "gemm_mxf4")


# ------------------------------------------------------------ torch helpers
class Mxf4Matrix:
    """A matrix [rows, k], or a batch [batch, rows, k], held in MXFP4 along k:
    ``codes`` and ``scales`` are the byte arrays include/gemm_mxf4.h lays out."""

    __slots__ = ("codes", "scales", "rows", "k", "batch")

    def __init__(self, codes, scales, rows: int, k: int, batch=None):
        self.codes, self.scales, self.rows, self.k, self.batch = codes, scales, rows, k, batch

    @property
    def shape(self):
        return (self.rows, self.k) if self.batch is None else (self.batch, self.rows, self.k)

    @property
    def device(self):
        return self.codes.device

    @property
    def nbytes(self) -> int:
        return self.codes.numel() + self.scales.numel()

    def __repr__(self):
        return f"Mxf4Matrix{self.shape} on {self.device}"


def _dtype_code(dtype) -> int:
    import torch

    code = {torch.float16: F16, torch.bfloat16: BF16, torch.float32: F32}.get(dtype)
    if code is None:
        raise TypeError("MXFP4 conversions take float16, bfloat16 or float32")
    return code


def _stream(device, stream):
    import torch

    return (stream if stream is not None else torch.cuda.current_stream(device)).cuda_stream


def _empty(shape, dtype, device, stream):
    """torch.empty for `stream`: what the allocator hands out is ordered with
    the stream that will write it, the current one unless one is given."""
    import torch

    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def mxf4_quantize(x, axis: int = -1, stream=None) -> Mxf4Matrix:
    """x (2-D, or 3-D with a leading batch; float16, bfloat16 or float32; any
    positive strides) in MXFP4 along `axis`, the one a product will contract: a
    weight [K, N] takes axis=-2 and becomes the [N, K] matrix that mxf4_mm and
    moe_few read."""
    import torch

    if x.dim() not in (2, 3):
        raise ValueError("mxf4_quantize takes a matrix or a batch of matrices")
    if axis not in (-1, -2, x.dim() - 1, x.dim() - 2):
        raise ValueError("axis must be one of the two matrix dimensions")
    code = _dtype_code(x.dtype)
    if not x.is_cuda:
        raise ValueError("tensors must be on a CUDA device")
    if axis % x.dim() == x.dim() - 2:
        x = x.transpose(-1, -2)
    rows, k = x.shape[-2:]
    batch = x.shape[0] if x.dim() == 3 else 1
    nc, ns = mxf4_sizes(rows, k, batch)
    codes = _empty(nc, torch.uint8, x.device, stream)
    scales = _empty(ns, torch.uint8, x.device, stream)
    with torch.cuda.device(x.device):
        # (a dimension of one element may carry any stride, a batch of stride 0 repeats)
        mxf4_quantize_ptr(x.data_ptr(), code, x.stride(0) if x.dim() == 3 and batch > 1 else 0,
                          x.stride(-2) if rows > 1 else max(1, k), x.stride(-1) if k > 1 else 1, codes.data_ptr(),
                          scales.data_ptr(), rows, k, batch, _stream(x.device, stream))
    return Mxf4Matrix(codes, scales, rows, k, batch if x.dim() == 3 else None)


def mxf4_dequantize(q: Mxf4Matrix, dtype=None, stream=None):
    """The values of q, rounded once to `dtype` (float16 unless given)."""
    import torch

    dtype = torch.float16 if dtype is None else dtype
    code = _dtype_code(dtype)
    y = _empty(q.shape, dtype, q.device, stream)
    with torch.cuda.device(q.device):
        mxf4_dequantize_ptr(q.codes.data_ptr(), q.scales.data_ptr(), y.data_ptr(), code, q.rows, q.k, q.batch or 1,
                            _stream(q.device, stream))
    return y


def mxf4_mm(a, b: Mxf4Matrix, bias=None, act="none", out=None, stream=None):
    """fp16 C[m, n] = act(sum_k a[m, k] b[n, k] + bias[n]): b an Mxf4Matrix
    [N, K], a an Mxf4Matrix [M, K] or a float16 tensor [M, K] that is quantised
    on the way; returns C."""
    import torch

    g = _pkg()
    if not isinstance(b, Mxf4Matrix) or b.batch is not None:
        raise TypeError("mxf4_mm takes b as an Mxf4Matrix of two dimensions")
    if isinstance(a, Mxf4Matrix):
        if a.batch is not None:
            raise ValueError("mxf4_mm takes matrices, not batches")
    elif a.dim() != 2:
        raise ValueError("expected two matrices")
    if a.shape[1] != b.k:
        raise ValueError(f"inner dimensions differ: {a.shape[1]} vs {b.k}")
    M, N = a.shape[0], b.rows
    code = g._act(act)
    if bias is not None and (bias.dim() != 1 or bias.shape[0] != N or bias.stride(0) != 1):
        raise ValueError("bias must hold N values with unit stride")
    g._check_out(out, (M, N), "[M, N]")
    g._check_tensors(None if isinstance(a, Mxf4Matrix) else a, out, bias)
    if any(t is not None and t.device != b.device for t in (a, out, bias)):
        raise ValueError("tensors must share one CUDA device")
    if out is None:
        out = _empty((M, N), torch.float16, b.device, stream)
    if not isinstance(a, Mxf4Matrix):
        a = mxf4_quantize(a, stream=stream)
    with torch.cuda.device(b.device):
        gemm_mxf4(a.codes.data_ptr(), a.scales.data_ptr(), b.codes.data_ptr(), b.scales.data_ptr(),
                  0 if bias is None else bias.data_ptr(), code, out.data_ptr(), out.stride(0), M, N, b.k,
                  _stream(b.device, stream))
    return out
