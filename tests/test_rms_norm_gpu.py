"""The norm against 64 bits.

h is exact (a sum of two 16-bit values rounded once).  A sum of d squares in fp32, eight values a lane
in order and then a tree, is off by at most (8 * vectors + 12) 2^-24 of itself, under 2^-18 with 4
vectors; the root halves that, and the quotient, the root and two products add four roundings: y is
within 2^-18 of itself before its own rounding (2^-11 of it in fp16, 2^-25 where it is subnormal; 2^-8 in
bf16).  In 8 bits: within half a step of the block's grid, 2^-4 of the value and 2^-10 of the scale,
where the scale is the definition's of y in 64 bits or, next to a border, its neighbour.
"""
import numpy as np
import pytest
import torch

import dense_tiled_gemm_fp16_gb300 as g
from tests.test_fp8_gpu import _arrays
from tests.fp8_reference import dequantize64, quantize64

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
TYPES = [torch.float16, torch.bfloat16]
SHAPES = [(1, 1), (1, 8), (3, 128), (5, 200), (300, 256), (77, 500), (9, 1024), (129, 1025), (16, 8192), (1, 8191), (400, 2048),
          (200, 3000), (300, 4097), (160, 7168), (1000, 8192), (3, 16384), (2, 20001), (2, 32768), (130, 640)]


def _inputs(rows, d, dtype, seed=0):
    gen = torch.Generator().manual_seed(rows + d + seed)
    x, r = (torch.randn((rows, d), generator=gen).mul_(s).to(dtype) for s in (1.0, 3.0))
    return x, r, (1 + 0.3 * torch.randn(d, generator=gen)).to(dtype)


def _reference(h, w, eps):
    h, w = h.double().numpy(), w.double().numpy()
    return h / np.sqrt((h * h).mean(axis=1, keepdims=True) + eps) * w


def _near(y, v):
    half = y.dtype is torch.float16
    tol = 2.0 ** -18 * np.abs(v) + (2.0 ** -11 * np.abs(v) + 2.0 ** -25 if half else 2.0 ** -8 * np.abs(v))
    err = np.abs(y.cpu().double().numpy() - v)
    assert (err <= tol * 1.001).all(), (err / tol).max()   # (a step's rounding is of the value as it was computed)


def _near_in_8_bits(q, v):
    (codes, scales), = _arrays(q)
    _, ref = quantize64(v)
    top = np.abs(np.pad(v, ((0, 0), (0, -v.shape[1] % 128)))).reshape(v.shape[0], -1, 128).max(-1)
    border = 448.0 * np.exp2(ref.astype(np.float64) - 127)   # the largest magnitude that has this scale
    beside = (np.abs(top / border - 1) < 2.0 ** -17) | (np.abs(2 * top / border - 1) < 2.0 ** -17)
    d = scales.astype(int) - ref
    assert (d[~beside] == 0).all() and (np.abs(d) <= 1).all()
    full = np.zeros((v.shape[0], scales.shape[1] * 128), np.uint8)
    full[:, :v.shape[1]] = codes
    got = dequantize64(full, scales)[:, :v.shape[1]]
    step = np.repeat(np.exp2(scales.astype(np.float64) - 127), 128, axis=1)[:, :v.shape[1]]
    tol = np.maximum(2.0 ** -4 * np.abs(v), 2.0 ** -10 * step) * (1 + 2.0 ** -3) + 2.0 ** -17 * np.abs(v)
    assert (np.abs(got - v) <= tol).all()
    # and nearly everywhere the value that 64 bits round to
    want = dequantize64(*quantize64(v))[:, :v.shape[1]]
    assert (got != want).mean() < 1e-4 or (got != want).sum() <= 1


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,d", SHAPES)
@pytest.mark.parametrize("residual", [False, True])
def test_against_64_bits(rows, d, residual, dtype):
    x, r, w = _inputs(rows, d, dtype)
    h = (x.float() + r.float()).to(dtype) if residual else x
    v = _reference(h, w, 1e-5)
    args = dict(eps=1e-5, residual=r.to(DEV) if residual else None)
    y = g.rms_norm(x.to(DEV), w.to(DEV), **args)
    q = g.rms_norm(x.to(DEV), w.to(DEV), quantize=True, **args)
    if residual:
        (y, s), (q, s2) = y, q
        assert torch.equal(s.cpu(), h) and torch.equal(s2.cpu(), h)
    _near(y, v)
    _near_in_8_bits(q, v)


@pytest.mark.parametrize("rows,d", [(3, 72), (40, 1030), (300, 7168), (2, 12000)])
def test_strides_places_and_in_place(rows, d):
    for dtype in TYPES:
        x, r, w = _inputs(rows, d, dtype)
        ref, href = g.rms_norm(x.to(DEV), w.to(DEV), residual=r.to(DEV))
        for lead, pitch in ((0, 8), (3, 5), (1, 0)):
            bufs = [torch.full((rows + 2, d + lead + pitch), -7.0, dtype=dtype, device=DEV) for _ in range(4)]
            vx, vr, vy, vs = (b[1:rows + 1, lead:lead + d] for b in bufs)
            vx.copy_(x)
            vr.copy_(r)
            y, h = g.rms_norm(vx, w.to(DEV), residual=vr, out=vy, sum_out=vs)
            assert y is vy and h is vs and torch.equal(vy, ref) and torch.equal(vs, href)
            for b, v in zip(bufs, (vx, vr, vy, vs)):
                v.fill_(-7.0)
                assert (b == -7.0).all()   # nothing around them was written
            for place in (vr, vx):
                vx.copy_(x)
                vr.copy_(r)
                y, h = g.rms_norm(vx, w.to(DEV), residual=vr, sum_out=place)
                assert torch.equal(y, ref) and torch.equal(place, href)


def test_rows_of_zeros_infinities_and_nans():
    for dtype in TYPES:
        x, _, w = _inputs(6, 400, dtype)
        x[1], x[2, 7], x[3, 399], x[4] = 0, float("inf"), float("nan"), 2.0 ** -20
        y = g.rms_norm(x.to(DEV), w.to(DEV)).cpu()
        assert (y[1] == 0).all() and y[2, 7].isnan() and y[3].isnan().all()
        assert not y[[0, 1, 4, 5]].isnan().any() and (y[2, :7] == 0).all()
        assert g.rms_norm(x[1:2].to(DEV), w.to(DEV), eps=0.0).isnan().all()   # 0 / 0
        back = g.fp8_dequantize(g.rms_norm(x.to(DEV), w.to(DEV), quantize=True)).cpu()
        assert back[2, :128].isnan().all() and not back[2, 128:].isnan().any() and back[3].isnan().all()
        assert not back[[0, 1, 4, 5]].isnan().any()


def test_no_rows_streams_and_graphs():
    x, r, w = (v.to(DEV) for v in _inputs(50, 3000, torch.float16))
    assert g.rms_norm(x[:0], w).shape == (0, 3000)
    ref, href = g.rms_norm(x, w, residual=r)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y, h = g.rms_norm(x, w, residual=r, stream=s)
    s.synchronize()
    assert torch.equal(y, ref) and torch.equal(h, href)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q, h = g.rms_norm(x, w, residual=r, quantize=True)
        y = g.fp8_dequantize(q)
    x.neg_(), r.neg_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(h, -href)
    assert torch.equal(y, g.fp8_dequantize(g.rms_norm(x, w, residual=r, quantize=True)[0]))
