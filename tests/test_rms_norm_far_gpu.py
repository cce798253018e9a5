"""The norm of bf16 rows whose squares fp32 does not hold, against 64 bits.

bf16 reaches from 2^-133 to 2^128, a square from 2^-266 to 2^256.  The sum of such a row is off by at
most 69 roundings (2^-17.9 of itself); the root halves that, the factor has 21 bits where it is subnormal
(2^-22), and the quotient, the root and three products add five roundings: together under 2^-18, as for every
other row.  Then y is rounded once (2^-8 of it in bf16, 2^-134 where it is subnormal), or in 8 bits is within half a
step of its block's grid (2^-4 of it, 2^-10 of the scale).
"""
import numpy as np
import pytest
import torch

import dense_tiled_gemm_fp16_gb300 as g
from tests.fp8_reference import dequantize64, quantize64
from tests.test_fp8_gpu import _arrays

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
MOST = torch.finfo(torch.bfloat16).max
SHAPES = [(9, 1), (9, 200), (9, 1000), (200, 512), (9, 1500), (200, 4097), (9, 7168), (200, 7168), (9, 12000)]


def _rows(rows, d, seed):
    """Rows of every size bf16 has, among them ordinary ones, and some of few large and many small values."""
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, d), generator=gen, dtype=torch.float64)
    powers = [120.0, -130.0, 0.0, 64.0, 70.0, -60.0, -70.0, -100.0, 126.0]
    x *= torch.exp2(torch.tensor([powers[i % len(powers)] for i in range(rows)], dtype=torch.float64))[:, None]
    x[3::9, 1::3] *= 2.0 ** -60
    x[0::9, 0] = MOST
    x[1::9, 0] = 2.0 ** -133
    return x.clamp(-MOST, MOST).bfloat16(), (1 + 0.3 * torch.randn(d, generator=gen)).bfloat16()


def _reference(h, w, eps):
    h = h.double().numpy()
    return h / np.sqrt((h * h).mean(axis=1, keepdims=True) + eps) * w.double().numpy()


def _check(y, q, v):
    err = np.abs(y.cpu().double().numpy() - v)
    tol = (2.0 ** -18 + 2.0 ** -8 * (1 + 2.0 ** -18)) * np.abs(v) + 2.0 ** -134
    assert (err <= tol).all(), (np.argwhere(err > tol)[:5], (err / tol).max())
    (codes, scales), = _arrays(q)
    _, ref = quantize64(v)
    top = np.abs(np.pad(v, ((0, 0), (0, -v.shape[1] % 128)))).reshape(v.shape[0], -1, 128).max(-1)
    border = 448.0 * np.exp2(ref.astype(np.float64) - 127)
    beside = (np.abs(top / border - 1) < 2.0 ** -17) | (np.abs(2 * top / border - 1) < 2.0 ** -17)
    off = scales.astype(int) - ref
    assert (off[~beside] == 0).all() and (np.abs(off) <= 1).all()
    full = np.zeros((v.shape[0], scales.shape[1] * 128), np.uint8)
    full[:, :v.shape[1]] = codes
    got = dequantize64(full, scales)[:, :v.shape[1]]
    step = np.repeat(np.exp2(scales.astype(np.float64) - 127), 128, axis=1)[:, :v.shape[1]]
    # (next to a border of the scale the step may be the larger one: half of it is 2^-3 of the value at most)
    half = np.where(np.repeat(beside, 128, axis=1)[:, :v.shape[1]], 2.0, 1.0) * np.maximum(2.0 ** -4 * np.abs(v), 2.0 ** -10 * step)
    assert (np.abs(got - v) <= half * (1 + 2.0 ** -16) + 2.0 ** -17 * np.abs(v)).all()


@pytest.mark.parametrize("eps", [0.0, 1e-30, 1e-5])
@pytest.mark.parametrize("rows,d", SHAPES)
def test_rows_whose_squares_fp32_does_not_hold(rows, d, eps):
    x, w = _rows(rows, d, rows + d)
    v = _reference(x, w, eps)
    _check(g.rms_norm(x.to(DEV), w.to(DEV), eps=eps), g.rms_norm(x.to(DEV), w.to(DEV), eps=eps, quantize=True), v)


@pytest.mark.parametrize("rows,d", [(9, 1000), (200, 4097), (9, 7168)])
def test_with_a_residual_in_other_places(rows, d):
    """h is read back where it was written, in place and apart, and rows beside keep their bits."""
    x, w = _rows(rows, d, 3)
    r, _ = _rows(rows, d, 4)
    r[r.abs() > MOST / 4] = 1.0   # (no infinite sums)
    x[x.abs() > MOST / 4] = -2.0 ** 126
    h = (x.float() + r.float()).bfloat16()
    v = _reference(h, w, 0.0)
    y, s = g.rms_norm(x.to(DEV), w.to(DEV), eps=0.0, residual=r.to(DEV))
    q, s2 = g.rms_norm(x.to(DEV), w.to(DEV), eps=0.0, residual=r.to(DEV), quantize=True)
    assert torch.equal(s.cpu(), h) and torch.equal(s2.cpu(), h)
    _check(y, q, v)
    for lead in (0, 3):
        buf = torch.full((rows + 2, d + 8), -7.0, dtype=torch.bfloat16, device=DEV)
        place, out = buf[1:rows + 1, lead:lead + d], torch.empty((rows, d), dtype=torch.bfloat16, device=DEV)
        place.copy_(x)
        g.rms_norm(place, w.to(DEV), eps=0.0, residual=r.to(DEV), sum_out=place, out=out)
        assert torch.equal(out, y) and torch.equal(place, s)
        place.fill_(-7.0)
        assert (buf == -7.0).all()


def test_a_far_row_has_the_same_bits_among_few_and_many():
    x, w = _rows(9, 7168, 5)
    y = g.rms_norm(x.to(DEV), w.to(DEV), eps=0.0)
    many = g.rms_norm(x.repeat(100, 1).to(DEV), w.to(DEV), eps=0.0)
    assert torch.equal(many, y.repeat(100, 1))
