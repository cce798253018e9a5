"""MXFP4 matrices on CUDA torch tensors: quantisation, its inverse and the product.

Mirrors ``include/gemm_mxf4.h`` (``mxf4_sizes``, ``gemm_mxf4``, ``gemm_mxf4_a16``
and the pointer forms of the two conversions) and adds the tensor forms
``mxf4_quantize``, ``mxf4_dequantize`` and ``mxf4_mm``.  Like the rest of the
binding it only marshals arguments; PyTorch supplies memory and streams.
"""
from __future__ import annotations

import ctypes

F16, BF16, F32 = range(3)

# Every symbol include/gemm_mxf4.h declares.
EXPORTED = ("mxf4_sizes", "mxf4_quantize", "mxf4_dequantize", "gemm_mxf4", "gemm_mxf4_a16")


def declare(L) -> None:
    """Argument types of the header's functions on the loaded library."""
    P, I64, I = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    L.mxf4_sizes.argtypes = [I64, I64, I64, ctypes.POINTER(I64), ctypes.POINTER(I64)]
    L.mxf4_quantize.argtypes = [P, I, I64, I64, I64, P, P, I64, I64, I64, P]
    L.mxf4_dequantize.argtypes = [P, P, P, I, I64, I64, I64, P]
    L.gemm_mxf4.argtypes = [P, P, P, P, P, I, P, I64, I64, I64, I64, P]
    L.gemm_mxf4_a16.argtypes = [P, I64, I64, P, P, P, P, I, P, I64, I64, I64, I64, P]
    for name in EXPORTED:
        getattr(L, name).restype = I


# The package and torch, looked up at the first call (the package imports this
# module, and its C mirrors work without torch), and what the tensor forms take
# from them: a call of a few microseconds is mostly Python otherwise.
_g = None
_t = None
_codes = {}   # torch dtype -> element type
_u8 = None    # torch.uint8
_device = None   # the current device's index
_raw = None   # the handle of a device's current stream
_fns = {}     # functions of the library that the tensor forms have called


def _pkg():
    global _g
    if _g is None:
        import dense_tiled_gemm_fp16_gb300 as g
        _g = g
    return _g


def _torch():
    global _t, _u8, _device, _raw
    if _t is None:
        import torch
        _codes.update({torch.float16: F16, torch.bfloat16: BF16, torch.float32: F32})
        _u8, _device, _raw = torch.uint8, torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
        _t = torch
    return _t


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


def gemm_mxf4_a16(A: int, stride_am: int, stride_ak: int, work: int, B_codes: int, B_scales: int, bias: int, act: int,
                  C: int, ldc: int, M: int, N: int, K: int, stream: int = 0) -> None:
    """gemm_mxf4 with A in fp16, quantised into `work` (see include/gemm_mxf4.h)."""
    g = _pkg()
    g._check(g.lib().gemm_mxf4_a16(A, stride_am, stride_ak, work, B_codes, B_scales, bias or None, act, C, ldc, M, N,
                                   K, stream or None), "gemm_mxf4_a16")


# ------------------------------------------------------------ torch helpers
def _bytes(rows: int, k: int, batch: int):
    """mxf4_sizes without its checks: (codes, scales)."""
    blocks = (k + 31) >> 5
    return batch * rows * blocks * 16, batch * ((rows + 127) >> 7) * ((blocks + 3) >> 2) * 512


class Mxf4Matrix:
    """A matrix [rows, k], or a batch [batch, rows, k], held in MXFP4 along k:
    ``codes`` and ``scales`` are the byte arrays include/gemm_mxf4.h lays out
    (contiguous uint8), ``codes_ptr`` and ``scales_ptr`` their device addresses."""

    __slots__ = ("_data", "_split", "rows", "k", "batch", "device", "codes_ptr", "scales_ptr")

    def __init__(self, codes, scales, rows: int, k: int, batch=None):
        u8 = (_t or _torch()).uint8
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
    def _of(cls, data, split: int, rows: int, k: int, batch, device):
        """Both arrays in one buffer, the codes from byte `split` on."""
        q = cls.__new__(cls)
        q._data, q._split = data, split
        q.rows, q.k, q.batch, q.device = rows, k, batch, device
        q.scales_ptr = p = data.data_ptr()
        q.codes_ptr = p + split
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
        return f"Mxf4Matrix{self.shape} on {self.device}"


def _dtype_code(dtype) -> int:
    _t or _torch()
    code = _codes.get(dtype)
    if code is None:
        raise TypeError("MXFP4 conversions take float16, bfloat16 or float32")
    return code


def _stream(device, stream) -> int:
    """Handle of `stream`, or of the device's current one."""
    return _raw(device.index) if stream is None else stream.cuda_stream


def _empty(shape, dtype, device, stream):
    """torch.empty for `stream`: what the allocator hands out is ordered with
    the stream that will write it, the current one unless one is given."""
    t = _t or _torch()
    if stream is None:
        return t.empty(shape, dtype=dtype, device=device)
    with t.cuda.stream(stream):
        return t.empty(shape, dtype=dtype, device=device)


def _run(device, name: str, *args) -> None:
    """The library's function `name` with `device` current; raises on a status
    that is not OK."""
    fn = _fns.get(name)
    if fn is None:
        fn = _fns[name] = getattr(_pkg().lib(), name)
    if device.index == _device():
        st = fn(*args)
    else:
        with _t.cuda.device(device):
            st = fn(*args)
    if st:
        _pkg()._check(st, name)


def _check_like(x, dtype, device, name: str) -> None:
    if x.dtype is not dtype:
        raise TypeError(f"mxf4_mm takes {name} as a float16 tensor")
    if x.device != device:
        raise ValueError("tensors must share one CUDA device")


def mxf4_quantize(x, axis: int = -1, stream=None) -> Mxf4Matrix:
    """x (2-D, or 3-D with a leading batch; float16, bfloat16 or float32; any
    positive strides) in MXFP4 along `axis`, the one a product will contract: a
    weight [K, N] takes axis=-2 and becomes the [N, K] matrix that mxf4_mm and
    moe_few read."""
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
        raise ValueError("mxf4_quantize takes a matrix or a batch of matrices")
    if axis == -2 or axis == nd - 2:
        rows, k, sr, sk = k, rows, sk, sr
    elif axis != -1 and axis != nd - 1:
        raise ValueError("axis must be one of the two matrix dimensions")
    code = _dtype_code(x.dtype)
    device = x.device
    if device.type != "cuda":
        raise ValueError("tensors must be on a CUDA device")
    nc, ns = _bytes(rows, k, batch)
    q = Mxf4Matrix._of(_empty(nc + ns, _u8, device, stream), ns, rows, k, held, device)
    # (a dimension of one element may carry any stride, a batch of stride 0 repeats)
    _run(device, "mxf4_quantize", x.data_ptr(), code, sb, sr if rows > 1 else max(1, k), sk if k > 1 else 1, q.codes_ptr,
         q.scales_ptr, rows, k, batch, _stream(device, stream))
    return q


def mxf4_dequantize(q: Mxf4Matrix, dtype=None, stream=None):
    """The values of q, rounded once to `dtype` (float16 unless given)."""
    if dtype is None:
        dtype = _torch().float16
    code = _dtype_code(dtype)
    device = q.device
    if device.type != "cuda":
        raise ValueError("tensors must be on a CUDA device")
    y = _empty(q.shape, dtype, device, stream)
    _run(device, "mxf4_dequantize", q.codes_ptr, q.scales_ptr, y.data_ptr(), code, q.rows, q.k, q.batch or 1,
         _stream(device, stream))
    return y


def mxf4_mm(a, b: Mxf4Matrix, bias=None, act="none", out=None, stream=None):
    """fp16 C[m, n] = act(sum_k a[m, k] b[n, k] + bias[n]): b an Mxf4Matrix
    [N, K], a an Mxf4Matrix [M, K] or a float16 tensor [M, K] that is quantised
    on the way; returns C."""
    if not isinstance(b, Mxf4Matrix) or b.batch is not None:
        raise TypeError("mxf4_mm takes b as an Mxf4Matrix of two dimensions")
    g, f16 = _g or _pkg(), (_t or _torch()).float16
    held = isinstance(a, Mxf4Matrix)
    shape = a.shape
    if len(shape) != 2:
        raise ValueError("expected two matrices")
    M, K = shape
    N, device = b.rows, b.device
    if K != b.k:
        raise ValueError(f"inner dimensions differ: {K} vs {b.k}")
    code = g._act(act)
    if not held and a.dtype is not f16:
        raise TypeError("mxf4_mm takes a as a float16 tensor or an Mxf4Matrix")
    if device.type != "cuda" or a.device != device:
        raise ValueError("tensors must share one CUDA device")
    bp = None
    if bias is not None:
        if bias.dim() != 1 or bias.shape[0] != N or bias.stride(0) != 1:
            raise ValueError("bias must hold N values with unit stride")
        _check_like(bias, f16, device, "bias")
        bp = bias.data_ptr()
    if out is None:
        out, ldc = _empty((M, N), f16, device, stream), N
    else:
        g._check_out(out, (M, N), "[M, N]")
        _check_like(out, f16, device, "out")
        ldc = out.stride(0) if M > 1 else N
    if held:
        _run(device, "gemm_mxf4", a.codes_ptr, a.scales_ptr, b.codes_ptr, b.scales_ptr, bp, code, out.data_ptr(), ldc, M,
             N, K, _stream(device, stream))
    else:
        sm, sk = a.stride()
        nc, ns = _bytes(M, K, 1)
        work = _empty(nc + ns, _u8, device, stream)
        _run(device, "gemm_mxf4_a16", a.data_ptr(), sm if M > 1 else max(1, K), sk if K > 1 else 1, work.data_ptr(),
             b.codes_ptr, b.scales_ptr, bp, code, out.data_ptr(), ldc, M, N, K, _stream(device, stream))
    return out
