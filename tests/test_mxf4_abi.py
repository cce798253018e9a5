"""The MXFP4 entry points without a GPU: exports, sizes and refusals."""
import ctypes
import os
import re

import pytest
import torch

import dense_tiled_gemm_fp16_gb300 as g
from dense_tiled_gemm_fp16_gb300 import mxf4

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# Fake, non-null, aligned "pointers": the calls are refused before any use.
X, C, S, Y = 1 << 20, 1 << 24, 1 << 28, 1 << 32


def _refused(call, status=g.ERR_INVALID_VALUE):
    with pytest.raises(g.GemmF16Error) as e:
        call()
    assert e.value.status == status


def test_every_declared_symbol_is_exported():
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "gemm_mxf4.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(\w*mxf4\w*)\s*\(", src))
    assert names == set(mxf4.EXPORTED)
    for n in names:
        assert ctypes.cast(getattr(g.lib(), n), ctypes.c_void_p).value
    for name, value in re.findall(r"MXF4_(\w+) = (\d)", src):
        assert getattr(mxf4, name) == int(value)


@pytest.mark.parametrize("rows,k,batch,codes,scales", [
    (1, 1, 1, 16, 512), (128, 128, 1, 128 * 64, 512), (129, 129, 1, 129 * 80, 4 * 512),
    (100, 4097, 3, 3 * 100 * 129 * 16, 3 * 33 * 512)])
def test_sizes(rows, k, batch, codes, scales):
    assert g.mxf4_sizes(rows, k, batch) == (codes, scales)


@pytest.mark.parametrize("args", [(0, 4, 1), (4, 0, 1), (4, 4, 0), (-1, 4, 1), (g.MAX_DIM + 1, 4, 1),
                                  (4, g.MAX_DIM + 1, 1), (g.MAX_DIM, g.MAX_DIM, 1 << 40)])
def test_sizes_refuses(args):
    _refused(lambda: g.mxf4_sizes(*args))


@pytest.mark.parametrize("args", [
    (0, 0, 0, 64, 1, C, S, 4, 64, 1),          # no input
    (X, 0, 0, 64, 1, 0, S, 4, 64, 1),          # no codes
    (X, 0, 0, 64, 1, C, 0, 4, 64, 1),          # no scales
    (X, 3, 0, 64, 1, C, S, 4, 64, 1),          # unknown type
    (X, 0, 0, 0, 1, C, S, 4, 64, 1),           # zero row stride
    (X, 0, 0, 64, -1, C, S, 4, 64, 1),         # negative stride
    (X, 0, -1, 64, 1, C, S, 4, 64, 2),         # negative batch stride
    (X + 1, 0, 0, 64, 1, C, S, 4, 64, 1),      # misaligned input
    (X + 2, 2, 0, 64, 1, C, S, 4, 64, 1),      # misaligned for fp32
    (X, 0, 0, 64, 1, C + 8, S, 4, 64, 1),      # misaligned codes
    (X, 0, 0, 64, 1, C, S + 4, 4, 64, 1),      # misaligned scales
    (X, 0, 0, 64, 1, C, S, 0, 64, 1),          # no rows
    (X, 0, 0, 64, 1, C, S, 4, 64, 65536),      # batch past the grid
    (X, 0, 0, 1 << 62, 1, C, S, 4, 64, 1),     # extent overflows
])
def test_quantize_refuses(args):
    _refused(lambda: g.mxf4_quantize_ptr(*args))


def test_overlaps_are_refused():
    _refused(lambda: g.mxf4_quantize_ptr(X, 0, 0, 64, 1, X + 256, S, 4, 64, 1), g.ERR_ALIAS)
    _refused(lambda: g.mxf4_quantize_ptr(X, 0, 0, 64, 1, C, X, 4, 64, 1), g.ERR_ALIAS)
    _refused(lambda: g.mxf4_quantize_ptr(X, 0, 0, 64, 1, C, C + 64, 4, 64, 1), g.ERR_ALIAS)
    _refused(lambda: g.mxf4_dequantize_ptr(C, S, C + 16, 0, 4, 64, 1), g.ERR_ALIAS)
    _refused(lambda: g.mxf4_dequantize_ptr(C, S, S + 16, 0, 4, 64, 1), g.ERR_ALIAS)
    for bad in (C, S, X, Y):
        _refused(lambda: g.gemm_mxf4(C, S, X, Y, 0, 0, bad, 8, 8, 8, 64), g.ERR_ALIAS)
    _refused(lambda: g.gemm_mxf4(C, S, X, Y, (1 << 36) + 2, 0, 1 << 36, 8, 8, 8, 64), g.ERR_ALIAS)


@pytest.mark.parametrize("args", [
    (0, S, X, Y, 0, 0, 1 << 36, 8, 8, 8, 64), (C, 0, X, Y, 0, 0, 1 << 36, 8, 8, 8, 64),
    (C, S, 0, Y, 0, 0, 1 << 36, 8, 8, 8, 64), (C, S, X, 0, 0, 0, 1 << 36, 8, 8, 8, 64),
    (C, S, X, Y, 0, 0, 0, 8, 8, 8, 64),               # no output
    (C, S, X, Y, 0, 4, 1 << 36, 8, 8, 8, 64),         # unknown activation
    (C, S, X, Y, 0, -1, 1 << 36, 8, 8, 8, 64),
    (C, S, X, Y, 0, 0, 1 << 36, 7, 8, 8, 64),         # ldc < N
    (C, S, X, Y, 0, 0, (1 << 36) + 1, 8, 8, 8, 64),   # misaligned C
    (C, S, X, Y, 3, 0, 1 << 36, 8, 8, 8, 64),         # misaligned bias
    (C + 8, S, X, Y, 0, 0, 1 << 36, 8, 8, 8, 64),     # misaligned codes
    (C, S, X, Y + 8, 0, 0, 1 << 36, 8, 8, 8, 64),     # misaligned scales
    (C, S, X, Y, 0, 0, 1 << 36, 8, 0, 8, 64), (C, S, X, Y, 0, 0, 1 << 36, 8, 8, 0, 64),
    (C, S, X, Y, 0, 0, 1 << 36, 8, 8, 8, 0),
])
def test_gemm_refuses(args):
    _refused(lambda: g.gemm_mxf4(*args))


@pytest.mark.parametrize("args", [
    (0, 64, 1, S, X, Y, 0, 0, 1 << 36, 8, 8, 8, 64), (C, 64, 1, 0, X, Y, 0, 0, 1 << 36, 8, 8, 8, 64),
    (C, 64, 1, S, 0, Y, 0, 0, 1 << 36, 8, 8, 8, 64), (C, 64, 1, S, X, 0, 0, 0, 1 << 36, 8, 8, 8, 64),
    (C, 64, 1, S, X, Y, 0, 0, 0, 8, 8, 8, 64),
    (C + 1, 64, 1, S, X, Y, 0, 0, 1 << 36, 8, 8, 8, 64),     # misaligned A
    (C, 64, 1, S + 8, X, Y, 0, 0, 1 << 36, 8, 8, 8, 64),     # misaligned work
    (C, 0, 1, S, X, Y, 0, 0, 1 << 36, 8, 8, 8, 64), (C, 64, -1, S, X, Y, 0, 0, 1 << 36, 8, 8, 8, 64),
    (C, 1 << 62, 1, S, X, Y, 0, 0, 1 << 36, 8, 8, 8, 64),    # extent overflows
    (C, 64, 1, S, X, Y, 0, 5, 1 << 36, 8, 8, 8, 64), (C, 64, 1, S, X, Y, 0, 0, 1 << 36, 4, 8, 8, 64),
])
def test_gemm_a16_refuses(args):
    _refused(lambda: g.gemm_mxf4_a16(*args))


def test_gemm_a16_overlaps_are_refused():
    call = lambda a=C, w=S, b=X, bs=Y, bias=0, c=1 << 36: g.gemm_mxf4_a16(a, 64, 1, w, b, bs, bias, 0, c, 8, 8, 8, 64)  # noqa: E731
    for bad in (dict(c=C), dict(c=S + 512), dict(w=C), dict(w=X), dict(w=Y), dict(bias=S + 16), dict(c=X), dict(c=Y)):
        _refused(lambda: call(**bad), g.ERR_ALIAS)


def test_valid_calls_reach_the_device_check():
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    _refused(lambda: g.mxf4_quantize_ptr(X, 0, 0, 64, 1, C, S, 4, 64, 1), g.ERR_UNSUPPORTED_DEVICE)
    _refused(lambda: g.mxf4_dequantize_ptr(C, S, Y, 0, 4, 64, 1), g.ERR_UNSUPPORTED_DEVICE)
    _refused(lambda: g.gemm_mxf4(C, S, X, Y, 0, 0, 1 << 36, 8, 8, 8, 64), g.ERR_UNSUPPORTED_DEVICE)
    _refused(lambda: g.gemm_mxf4_a16(C, 64, 1, S, X, Y, 0, 0, 1 << 36, 8, 8, 8, 64), g.ERR_UNSUPPORTED_DEVICE)


def test_tensor_forms_check_before_any_call():
    h = torch.float16
    with pytest.raises(TypeError):
        g.mxf4_quantize(torch.zeros((4, 64), dtype=torch.float64))
    with pytest.raises(ValueError):                      # host tensor
        g.mxf4_quantize(torch.zeros((4, 64), dtype=h))
    with pytest.raises(ValueError):
        g.mxf4_quantize(torch.zeros(64, dtype=h))
    with pytest.raises(ValueError):
        g.mxf4_quantize(torch.zeros((4, 4, 64), dtype=h), axis=0)
    q = g.Mxf4Matrix(torch.zeros(4 * 32, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8), 4, 64)
    with pytest.raises(TypeError):
        g.mxf4_dequantize(q, torch.int8)
    a = torch.zeros((3, 64), dtype=h)
    with pytest.raises(ValueError):                      # arrays of other sizes
        g.Mxf4Matrix(torch.zeros(128, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8), 5, 64)
    with pytest.raises(TypeError):                       # b must be quantised
        g.mxf4_mm(a, a)
    with pytest.raises(ValueError):                      # inner dimensions
        g.mxf4_mm(a[:, :32], q)
    with pytest.raises(ValueError):
        g.mxf4_mm(a, q, act="tanh")
    with pytest.raises(ValueError):
        g.mxf4_mm(a, q, bias=torch.zeros(3, dtype=h))
    with pytest.raises(ValueError):
        g.mxf4_mm(a, q, out=torch.zeros((3, 5), dtype=h))
    with pytest.raises(TypeError):
        g.mxf4_mm(a.float(), q)
    with pytest.raises(ValueError):                      # host tensors
        g.mxf4_mm(a, q)
    batch = g.Mxf4Matrix(q.codes, q.scales, 4, 64, 1)
    with pytest.raises(TypeError):
        g.mxf4_mm(a, batch)
    with pytest.raises(ValueError):
        g.mxf4_mm(batch, q)
