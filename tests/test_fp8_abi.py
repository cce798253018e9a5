"""The 8-bit products, the norm and the expert order without a GPU: exports, sizes and refusals."""
import ctypes
import os
import re

import pytest
import torch

import dense_tiled_gemm_fp16_gb300 as g
from dense_tiled_gemm_fp16_gb300 import fp8, norm, route

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# Fake, non-null, aligned "pointers": the calls are refused before any use.
X, C, S, Y, Z, W = 1 << 20, 1 << 24, 1 << 28, 1 << 32, 1 << 36, 1 << 40


def _refused(call, status=g.ERR_INVALID_VALUE):
    with pytest.raises(g.GemmF16Error) as e:
        call()
    assert e.value.status == status


def _changed(args, **by_place):
    out = list(args)
    for place, value in by_place.items():
        out[int(place[1:])] = value
    return out


@pytest.mark.parametrize("header,module", [("gemm_fp8.h", fp8), ("rms_norm.h", norm), ("moe_route.h", route)])
def test_every_declared_symbol_is_exported(header, module):
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header)).read(), flags=re.S)
    names = set(re.findall(r"^gemm_f16_status (\w+)\(", src, flags=re.M))
    assert names == set(module.EXPORTED)
    for n in names:
        assert ctypes.cast(getattr(g.lib(), n), ctypes.c_void_p).value
        assert getattr(g.lib(), n).argtypes
    for name, value in re.findall(r"#define \w+_(MAX_\w+) (\d+)", src):
        assert getattr(module, name) == int(value)
    for name, value in re.findall(r"FP8_(\w+) = (\d)", src):
        assert getattr(module, name) == int(value)


@pytest.mark.parametrize("rows,k,batch,codes,scales", [
    (1, 1, 1, 128, 512), (128, 512, 1, 128 * 512, 512), (129, 513, 1, 129 * 640, 4 * 512),
    (100, 4097, 3, 3 * 100 * 4224, 3 * 9 * 512)])
def test_sizes(rows, k, batch, codes, scales):
    assert g.fp8_sizes(rows, k, batch) == (codes, scales) == fp8._bytes(rows, k, batch)


@pytest.mark.parametrize("args", [(0, 4, 1), (4, 0, 1), (4, 4, 0), (-1, 4, 1), (g.MAX_DIM + 1, 4, 1),
                                  (4, g.MAX_DIM + 1, 1), (g.MAX_DIM, g.MAX_DIM, 1 << 40)])
def test_sizes_refuses(args):
    _refused(lambda: g.fp8_sizes(*args))


@pytest.mark.parametrize("args", [
    (0, 0, 0, 64, 1, C, S, 4, 64, 1), (X, 0, 0, 64, 1, 0, S, 4, 64, 1), (X, 0, 0, 64, 1, C, 0, 4, 64, 1),
    (X, 3, 0, 64, 1, C, S, 4, 64, 1),          # unknown type
    (X, 0, 0, 0, 1, C, S, 4, 64, 1), (X, 0, 0, 64, -1, C, S, 4, 64, 1), (X, 0, -1, 64, 1, C, S, 4, 64, 2),
    (X + 1, 0, 0, 64, 1, C, S, 4, 64, 1), (X + 2, 2, 0, 64, 1, C, S, 4, 64, 1),
    (X, 0, 0, 64, 1, C + 8, S, 4, 64, 1), (X, 0, 0, 64, 1, C, S + 4, 4, 64, 1),
    (X, 0, 0, 64, 1, C, S, 0, 64, 1), (X, 0, 0, 64, 1, C, S, 4, 64, 65536), (X, 0, 0, 1 << 62, 1, C, S, 4, 64, 1),
])
def test_quantize_refuses(args):
    _refused(lambda: g.fp8_quantize_ptr(*args))


def test_conversions_refuse_overlaps_and_types():
    _refused(lambda: g.fp8_quantize_ptr(X, 0, 0, 64, 1, X + 256, S, 4, 64, 1), g.ERR_ALIAS)
    _refused(lambda: g.fp8_quantize_ptr(X, 0, 0, 64, 1, C, X, 4, 64, 1), g.ERR_ALIAS)
    _refused(lambda: g.fp8_quantize_ptr(X, 0, 0, 64, 1, C, C + 64, 4, 64, 1), g.ERR_ALIAS)
    _refused(lambda: g.fp8_dequantize_ptr(C, S, C + 16, 0, 4, 64, 1), g.ERR_ALIAS)
    _refused(lambda: g.fp8_dequantize_ptr(C, S, S + 16, 0, 4, 64, 1), g.ERR_ALIAS)
    for args in ((0, S, X, 0, 4, 64, 1), (C, 0, X, 0, 4, 64, 1), (C, S, 0, 0, 4, 64, 1), (C, S, X, 3, 4, 64, 1),
                 (C, S, X + 1, 0, 4, 64, 1), (C, S, X, 0, 0, 64, 1), (C, S, X, 0, 4, 64, 70000)):
        _refused(lambda: g.fp8_dequantize_ptr(*args))


# A codes, A scales, B codes, B scales, bias, act, C, dtype, ldc, M, N, K
MM = (C, S, X, Y, 0, 0, Z, 0, 8, 8, 8, 64)


@pytest.mark.parametrize("change", [
    dict(_0=0), dict(_1=0), dict(_2=0), dict(_3=0), dict(_6=0), dict(_5=4), dict(_5=-1), dict(_7=2), dict(_7=-1),
    dict(_8=7), dict(_6=Z + 1), dict(_4=3), dict(_0=C + 8), dict(_3=Y + 8), dict(_9=0), dict(_10=0), dict(_11=0),
    dict(_9=-3), dict(_9=g.MAX_DIM + 1), dict(_8=1 << 62)])
def test_product_refuses(change):
    _refused(lambda: g.gemm_fp8(*_changed(MM, **change)))


# A, type, strides, work, B codes, B scales, bias, act, C, dtype, ldc, M, N, K
MM16 = (C, 0, 64, 1, S, X, Y, 0, 0, Z, 0, 8, 8, 8, 64)


@pytest.mark.parametrize("change", [
    dict(_0=0), dict(_0=C + 1), dict(_1=2), dict(_1=-1), dict(_2=0), dict(_3=-1), dict(_2=1 << 62), dict(_4=0), dict(_4=S + 8),
    dict(_5=0), dict(_6=0), dict(_9=0), dict(_8=9), dict(_10=2), dict(_11=4), dict(_12=0)])
def test_product_of_16_bit_rows_refuses(change):
    _refused(lambda: g.gemm_fp8_a16(*_changed(MM16, **change)))


# A codes, A scales, B codes, B scales, B_up codes, B_up scales, group_rows, act, C, dtype, ldc, rows, groups, N, K
GROUPED = (C, S, X, Y, 0, 0, W, 0, Z, 0, 8, 8, 4, 8, 64)
GROUPED16 = (C, 0, 64, 1, S, X, Y, 0, 0, W, 0, Z, 0, 8, 8, 4, 8, 64)


@pytest.mark.parametrize("change", [
    dict(_0=0), dict(_1=0), dict(_2=0), dict(_3=0), dict(_4=1 << 44), dict(_5=1 << 44), dict(_6=0), dict(_6=W + 2),
    dict(_7=4), dict(_8=0), dict(_9=2), dict(_10=7), dict(_11=-1), dict(_12=0), dict(_12=-1), dict(_12=513), dict(_13=0),
    dict(_14=0), dict(_14=g.MAX_DIM + 1), dict(_13=g.MAX_DIM, _12=512, _14=1 << 20)])
def test_grouped_product_refuses(change):
    _refused(lambda: g.gemm_fp8_grouped(*_changed(GROUPED, **change)))


@pytest.mark.parametrize("change", [dict(_0=0), dict(_1=2), dict(_2=0), dict(_4=0), dict(_5=0), dict(_9=0), dict(_14=-1),
                                    dict(_15=0)])
def test_grouped_product_of_16_bit_rows_refuses(change):
    _refused(lambda: g.gemm_fp8_grouped_a16(*_changed(GROUPED16, **change)))


def test_products_refuse_overlaps():
    for bad in (C, S, X, Y):
        _refused(lambda: g.gemm_fp8(*_changed(MM, _6=bad)), g.ERR_ALIAS)
    _refused(lambda: g.gemm_fp8(*_changed(MM, _4=Z + 2)), g.ERR_ALIAS)
    for bad in (C, X, Y, Z):
        _refused(lambda: g.gemm_fp8_a16(*_changed(MM16, _4=bad)), g.ERR_ALIAS)
    for bad in (C, S, X, Y, W):
        _refused(lambda: g.gemm_fp8_grouped(*_changed(GROUPED, _8=bad)), g.ERR_ALIAS)
    _refused(lambda: g.gemm_fp8_grouped(*_changed(GROUPED, _4=Z, _5=1 << 44)), g.ERR_ALIAS)
    _refused(lambda: g.gemm_fp8_grouped_a16(*_changed(GROUPED16, _9=S)), g.ERR_ALIAS)


def test_a_grouped_product_of_no_rows_is_done():
    g.gemm_fp8_grouped(0, 0, X, Y, 0, 0, W, 0, 0, 0, 8, 0, 4, 8, 64)
    g.gemm_fp8_grouped_a16(0, 0, 64, 1, 0, X, Y, 0, 0, W, 0, 0, 0, 8, 0, 4, 8, 64)


# x, dtype, stride, residual, stride, weight, eps, sum, stride, y, stride, codes, scales, rows, d
NORM = (X, 0, 64, C, 64, S, 1e-6, Y, 64, Z, 64, 0, 0, 4, 64)


@pytest.mark.parametrize("change", [
    dict(_0=0), dict(_0=X + 1), dict(_1=2), dict(_1=-1), dict(_2=63), dict(_4=63), dict(_8=63), dict(_10=63), dict(_5=0),
    dict(_5=S + 1), dict(_6=-1.0), dict(_6=float("nan")), dict(_6=float("inf")), dict(_7=0), dict(_3=0), dict(_9=0),
    dict(_11=W, _12=W + 4096), dict(_9=0, _11=W), dict(_9=0, _12=W), dict(_9=0, _11=W + 8, _12=1 << 44), dict(_13=-1),
    dict(_13=g.MAX_DIM + 1), dict(_14=0), dict(_14=norm.MAX_DIM + 1, _2=1 << 20, _4=1 << 20, _8=1 << 20, _10=1 << 20),
    dict(_2=1 << 62)])
def test_norm_refuses(change):
    _refused(lambda: g.rms_norm_ptr(*_changed(NORM, **change)))


def test_norm_refuses_overlaps():
    for bad in (X, C, S, Y):
        _refused(lambda: g.rms_norm_ptr(*_changed(NORM, _9=bad)), g.ERR_ALIAS)
    _refused(lambda: g.rms_norm_ptr(*_changed(NORM, _7=S)), g.ERR_ALIAS)
    _refused(lambda: g.rms_norm_ptr(*_changed(NORM, _7=X + 2)), g.ERR_ALIAS)          # neither in place nor apart
    _refused(lambda: g.rms_norm_ptr(*_changed(NORM, _7=C, _8=72)), g.ERR_ALIAS)
    for codes, scales in ((X, W), (W, X), (W, W), (Y, W)):
        _refused(lambda: g.rms_norm_ptr(*_changed(NORM, _9=0, _11=codes, _12=scales)), g.ERR_ALIAS)
    g.rms_norm_ptr(0, 0, 64, 0, 0, 0, 1e-6, 0, 0, 0, 0, 0, 0, 0, 64)                  # no rows: done


def test_order_refuses():
    assert g.moe_sort_workspace_size(16, 8, 64) == 0
    assert g.moe_sort_workspace_size(16384, 8, 64) == 128 * 65 * 4
    for args in ((-1, 8, 64), (16, 0, 64), (16, 33, 64), (16, 8, 0), (16, 8, 513), (g.MAX_DIM, 8, 64)):
        _refused(lambda: g.moe_sort_workspace_size(*args))
    sort = (X, 16, 8, 64, C, S, Y, 0, 0)
    for change in (dict(_0=0), dict(_4=0), dict(_5=0), dict(_6=0), dict(_0=X + 2), dict(_6=Y + 1), dict(_1=-1), dict(_2=0),
                   dict(_3=0), dict(_3=513)):
        _refused(lambda: g.moe_sort_ptr(*_changed(sort, **change)))
    for change in (dict(_4=X), dict(_5=X), dict(_6=X), dict(_5=C), dict(_6=C), dict(_6=S)):
        _refused(lambda: g.moe_sort_ptr(*_changed(sort, **change)), g.ERR_ALIAS)
    large = (X, 16384, 8, 64, C, S, Y, Z, 128 * 65 * 4)
    for change in (dict(_7=0), dict(_8=1000), dict(_7=Z + 128)):
        _refused(lambda: g.moe_sort_ptr(*_changed(large, **change)), g.ERR_OUT_OF_MEMORY)
    _refused(lambda: g.moe_sort_ptr(*_changed(large, _7=X)), g.ERR_ALIAS)


ROWS = {   # the call, its arguments, the places of: type, strides, rows, tokens, top_k, d; and pairs that may not overlap
    "moe_gather_ptr": ((X, 0, 64, C, 4, 2, 64, Y, 64), 1, (2, 8), 3, 4, 5, 6, ((7, X), (7, C))),
    "moe_combine_ptr": ((X, 0, 64, C, S, 4, 2, 64, Y, 64), 1, (2, 9), 3, 5, 6, 7, ((8, X), (8, C), (8, S))),
    "moe_combine_grad_ptr": ((X, 0, 64, Z, 64, C, S, 4, 2, 64, Y, 64, W), 1, (2, 4, 11), 5, 7, 8, 9,
                             ((10, X), (10, Z), (10, C), (10, S), (12, X), (12, C), (12, S), (12, Y))),
}


@pytest.mark.parametrize("name", ROWS)
def test_rows_refuse(name):
    args, dtype, strides, rows, tokens, top, d, clashes = ROWS[name]
    call = getattr(g, name)
    bad = [(0, 0), (0, X + 1), (dtype, 2), (dtype, -1), (rows, 0), (rows, C + 2), (tokens, -1), (top, 0), (top, 33), (d, 0),
           (tokens, g.MAX_DIM)] + [(s, 63) for s in strides] + [(s, 1 << 62) for s in strides]
    for place, value in bad:
        _refused(lambda: call(*_changed(args, **{f"_{place}": value})))
    for place, value in clashes:
        _refused(lambda: call(*_changed(args, **{f"_{place}": value})), g.ERR_ALIAS)
    call(*_changed(args, **{f"_{tokens}": 0, f"_{rows}": 0, "_0": 0}))   # no tokens: done


def test_8_bit_rows_refuse():
    args = (X, C, S, 4, 2, 64, Y, Z)
    for change in (dict(_0=0), dict(_1=0), dict(_2=0), dict(_6=0), dict(_7=0), dict(_0=X + 8), dict(_7=Z + 4), dict(_3=-1),
                   dict(_4=0), dict(_5=0)):
        _refused(lambda: g.moe_gather_fp8_ptr(*_changed(args, **change)))
    for change in (dict(_6=X), dict(_6=C), dict(_7=X), dict(_7=S), dict(_7=Y)):
        _refused(lambda: g.moe_gather_fp8_ptr(*_changed(args, **change)), g.ERR_ALIAS)


# ------------------------------------------------------------ the tensor forms
def _held(rows, k, batch=None):
    nc, ns = fp8._bytes(rows, k, batch or 1)
    return g.Fp8Matrix(torch.zeros(nc, dtype=torch.uint8), torch.zeros(ns, dtype=torch.uint8), rows, k, batch)


H, B16 = torch.float16, torch.bfloat16


def z(*s, dtype=H):
    return torch.zeros(s, dtype=dtype)


def test_matrix():
    q = _held(3, 130, 2)
    assert q.shape == (2, 3, 130) and q.nbytes == sum(fp8._bytes(3, 130, 2)) and "Fp8Matrix" in repr(q)
    c, s = q.codes, q.scales
    with pytest.raises(TypeError):
        g.Fp8Matrix(c.char(), s, 3, 130, 2)
    with pytest.raises(ValueError, match="hold"):
        g.Fp8Matrix(c[1:], s, 3, 130, 2)
    with pytest.raises(ValueError, match="at least one"):
        g.Fp8Matrix(c, s, 0, 130, 2)
    with pytest.raises(ValueError, match="contiguous"):
        g.Fp8Matrix(torch.zeros(2 * c.numel(), dtype=torch.uint8)[::2], s, 3, 130, 2)


@pytest.mark.parametrize("call,error,match", [
    (lambda: g.fp8_quantize(z(4, 64)), ValueError, "CUDA"),
    (lambda: g.fp8_quantize(z(4)), ValueError, "matrix"),
    (lambda: g.fp8_quantize(z(4, 64), axis=0 - 3), ValueError, "axis"),
    (lambda: g.fp8_quantize(z(4, 64, dtype=torch.float64)), TypeError, "x must be"),
    (lambda: g.fp8_dequantize(_held(4, 64)), ValueError, "CUDA"),
    (lambda: g.fp8_dequantize(z(4, 64)), TypeError, "Fp8Matrix"),
    (lambda: g.fp8_dequantize(_held(4, 64), dtype=torch.int8), TypeError, "dtype must be"),
    (lambda: g.fp8_mm(z(4, 64), z(64, 4)), TypeError, "b as an Fp8Matrix"),
    (lambda: g.fp8_mm(z(4, 64), _held(4, 64, 2)), TypeError, "two dimensions"),
    (lambda: g.fp8_mm(z(4, 60), _held(4, 64)), ValueError, "inner"),
    (lambda: g.fp8_mm(z(4, 64, dtype=torch.float32), _held(4, 64)), TypeError, "a must be"),
    (lambda: g.fp8_mm(_held(4, 64, 1), _held(4, 64)), ValueError, "matrix"),
    (lambda: g.fp8_mm(z(4, 64), _held(4, 64)), ValueError, "CUDA"),
    (lambda: g.fp8_grouped_mm(z(4, 64), _held(4, 64), z(2, dtype=torch.int32)), TypeError, "batch"),
    (lambda: g.fp8_grouped_mm(z(4, 60), _held(4, 64, 2), z(2, dtype=torch.int32)), ValueError, "inner"),
    (lambda: g.fp8_grouped_mm(z(4, 64), _held(4, 64, 2), z(2, dtype=torch.int32), b_up=_held(3, 64, 2)), TypeError, "b_up"),
    (lambda: g.rms_norm(z(4), z(4)), ValueError, "rows, d"),
    (lambda: g.rms_norm(z(4, 8, dtype=torch.float32), z(8, dtype=torch.float32)), TypeError, "x must be"),
    (lambda: g.rms_norm(z(4, 8), z(7)), ValueError, "weight"),
    (lambda: g.rms_norm(z(4, 8), z(8, dtype=B16)), ValueError, "weight"),
    (lambda: g.rms_norm(z(8, 4).t(), z(8)), ValueError, "contiguous rows"),
    (lambda: g.rms_norm(z(4, 8), z(8)), ValueError, "CUDA"),
    (lambda: g.moe_sort(z(4, 2, dtype=torch.int64), 8), TypeError, "int32"),
    (lambda: g.moe_sort(z(4, 2, dtype=torch.int32), 8), ValueError, "CUDA"),
    (lambda: g.moe_gather(z(4, 8), g.MoeOrder(z(4, 2), None, None)), TypeError, "int32"),
    (lambda: g.moe_gather(z(4, 8), g.MoeOrder(z(4, 2, dtype=torch.int32), None, None)), ValueError, "CUDA"),
    (lambda: g.moe_combine(z(8, 8), g.MoeOrder(z(4, 2, dtype=torch.int32), None, None)), ValueError, "CUDA"),
])
def test_tensor_forms_refuse(call, error, match):
    with pytest.raises(error, match=match):
        call()


def on(*s, dtype=H):
    return torch.zeros(s, dtype=dtype, device="cuda:0")


@pytest.mark.gpu
@pytest.mark.parametrize("call,error,match", [
    (lambda q, o: g.fp8_quantize(on(4, 0)), ValueError, "at least one"),
    (lambda q, o: g.fp8_mm(on(4, 64), q, bias=on(5)), ValueError, "bias"),
    (lambda q, o: g.fp8_mm(on(4, 64), q, bias=on(6, dtype=B16)), TypeError, "bias"),
    (lambda q, o: g.fp8_mm(on(4, 64), q, bias=z(6)), ValueError, "device"),
    (lambda q, o: g.fp8_mm(z(4, 64), q), ValueError, "device"),
    (lambda q, o: g.fp8_mm(on(4, 64), q, dtype=torch.float32), TypeError, "dtype"),
    (lambda q, o: g.fp8_mm(on(4, 64), q, out=on(4, 6), dtype=B16), TypeError, "out"),
    (lambda q, o: g.fp8_mm(on(4, 64), q, out=on(4, 7)), ValueError, "out"),
    (lambda q, o: g.fp8_mm(on(4, 64), q, out=on(6, 4).t()), ValueError, "out"),
    (lambda q, o: g.fp8_mm(on(4, 64), q, out=z(4, 6)), ValueError, "device"),
    (lambda q, o: g.fp8_mm(on(4, 64), q, act="tanh"), ValueError, "activation"),
    (lambda q, o: g.fp8_mm(on(4, 64).expand(4, 64)[:, :1].expand(4, 64), q), g.GemmF16Error, "INVALID"),
    (lambda q, o: g.rms_norm(on(4, 8), on(8), residual=on(4, 7)), ValueError, "residual"),
    (lambda q, o: g.rms_norm(on(4, 8), on(8), residual=z(4, 8)), ValueError, "device"),
    (lambda q, o: g.rms_norm(on(4, 8), on(8), sum_out=on(4, 8)), ValueError, "sum_out"),
    (lambda q, o: g.rms_norm(on(4, 8), on(8), out=on(4, 8), quantize=True), ValueError, "out"),
    (lambda q, o: g.rms_norm(on(4, 8), on(8), eps=-1.0), g.GemmF16Error, "INVALID"),
    (lambda q, o: g.rms_norm(on(2, norm.MAX_DIM + 1), on(norm.MAX_DIM + 1)), g.GemmF16Error, "INVALID"),
    (lambda q, o: g.rms_norm(on(1, 8).expand(4, 8), on(8)), g.GemmF16Error, "INVALID"),
    (lambda q, o: g.moe_sort(on(4, 33, dtype=torch.int32), 8), g.GemmF16Error, "INVALID"),
    (lambda q, o: g.moe_sort(on(4, 2, dtype=torch.int32), 513), g.GemmF16Error, "INVALID"),
    (lambda q, o: g.moe_gather(on(5, 8), o), ValueError, "row for each token"),
    (lambda q, o: g.moe_gather(on(4, 8), o, out=on(7, 8)), ValueError, "out"),
    (lambda q, o: g.moe_combine(on(7, 8), o), ValueError, "row for each choice"),
    (lambda q, o: g.moe_combine(on(8, 8), o, on(4, 2)), TypeError, "weights"),
    (lambda q, o: g.moe_combine(on(8, 8), o, z(4, 2, dtype=torch.float32)), ValueError, "device"),
    (lambda q, o: g.moe_combine_grad(on(4, 7), on(8, 8), o, on(4, 2, dtype=torch.float32)), ValueError, "dout"),
    (lambda q, o: g.moe_combine_grad(on(4, 8, dtype=B16), on(8, 8), o, on(4, 2, dtype=torch.float32)), ValueError, "dout"),
])
def test_tensor_forms_refuse_on_the_device(call, error, match):
    q = g.fp8_quantize(on(6, 64))
    o = g.moe_sort(on(4, 2, dtype=torch.int32), 3)
    with pytest.raises(error, match=match):
        call(q, o)


@pytest.mark.gpu
def test_grouped_product_refuses_on_the_device():
    q = g.fp8_quantize(on(2, 6, 64))
    for counts, error in ((on(3, dtype=torch.int32), TypeError), (on(2, dtype=torch.int64), TypeError),
                          (z(2, dtype=torch.int32), ValueError), (on(4, dtype=torch.int32)[::2], ValueError)):
        with pytest.raises(error):
            g.fp8_grouped_mm(on(4, 64), q, counts)
    with pytest.raises(g.GemmF16Error):
        many = g.fp8_quantize(on(513, 1, 64))
        g.fp8_grouped_mm(on(4, 64), many, on(513, dtype=torch.int32))
