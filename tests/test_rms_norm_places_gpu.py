"""The norm with x, residual, sum, y and weight each at a place and a pitch of its own.

The values are those of the same call on contiguous tensors, bit for bit: neither the sum's order nor a rounding
hangs on where rows lie.  That call is compared with 64 bits elsewhere.
"""
import itertools

import pytest
import torch

import dense_tiled_gemm_fp16_gb300 as g

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
TYPES = [torch.float16, torch.bfloat16]
# a warp a row (up to 1024 values), a block a row of each form, few rows and many
SHAPES = [(5, 72), (40, 200), (300, 500), (40, 1000), (300, 1030), (3, 2056), (200, 2056), (200, 4097), (300, 7168), (3, 7168),
          (2, 12000), (170, 12000)]
# values before the first row's start, and between rows, of x, residual, sum, y and weight
PLACES = [((0, 0), (3, 5), (5, 3), (1, 7), (2, 0)), ((3, 5), (0, 8), (0, 0), (0, 0), (0, 0)), ((0, 8), (0, 8), (1, 0), (8, 8), (0, 0)),
          ((7, 1), (6, 2), (6, 2), (3, 6), (8, 0)), ((1, 3), (1, 3), (2, 5), (1, 3), (7, 0)), ((8, 8), (8, 0), (0, 8), (8, 8), (1, 0))]


def _place(v, lead, pitch):
    """v inside a buffer of -7, and the buffer."""
    rows, d = v.shape
    buf = torch.full((rows + 2, d + lead + pitch), -7.0, dtype=v.dtype, device=DEV)
    at = buf[1:rows + 1, lead:lead + d]
    at.copy_(v)
    return at, buf


def _inputs(rows, d, dtype):
    gen = torch.Generator().manual_seed(rows + d)
    x, r = (torch.randn((rows, d), generator=gen).mul_(s).to(dtype).to(DEV) for s in (1.0, 3.0))
    return x, r, (1 + 0.3 * torch.randn(d, generator=gen)).to(dtype).to(DEV)


def _clean(*pairs):
    for v, buf in pairs:
        v.fill_(-7.0)
        assert (buf == -7.0).all()   # nothing around it was written


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,d", SHAPES)
def test_each_at_a_place_of_its_own(rows, d, dtype):
    x, r, w = _inputs(rows, d, dtype)
    ref, href = g.rms_norm(x, w, residual=r)
    alone, qref = g.rms_norm(x, w), g.rms_norm(x, w, residual=r, quantize=True)[0]
    for px, pr, ps, py, pw in PLACES:
        vx, bx = _place(x, *px)
        vr, br = _place(r, *pr)
        vs, bs = _place(torch.zeros_like(x), *ps)
        vy, by = _place(torch.zeros_like(x), *py)
        vw = _place(w[None], *pw)[0][0]
        g.rms_norm(vx, vw, residual=vr, out=vy, sum_out=vs)
        assert torch.equal(vy, ref) and torch.equal(vs, href) and torch.equal(vx, x) and torch.equal(vr, r)
        vs.zero_()
        q, _ = g.rms_norm(vx, vw, residual=vr, quantize=True, sum_out=vs)
        assert torch.equal(q.codes, qref.codes) and torch.equal(q.scales, qref.scales) and torch.equal(vs, href)
        g.rms_norm(vx, vw, out=vy)
        assert torch.equal(vy, alone)
        _clean((vx, bx), (vr, br), (vs, bs), (vy, by))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,d", SHAPES)
def test_in_place_with_unlike_starts(rows, d, dtype):
    """The sum over x or over the residual while the other one starts elsewhere: threads of a row write what
    others have read."""
    x, r, w = _inputs(rows, d, dtype)
    ref, href = g.rms_norm(x, w, residual=r)
    qref = g.rms_norm(x, w, residual=r, quantize=True)[0]
    for px, pr in itertools.permutations(((0, 0), (3, 5), (5, 2), (8, 8), (1, 0)), 2):
        for over in (0, 1):
            for quantize in (False, True):
                (vx, bx), (vr, br) = _place(x, *px), _place(r, *pr)
                y, h = g.rms_norm(vx, w, residual=vr, sum_out=(vx, vr)[over], quantize=quantize)
                assert h is (vx, vr)[over] and torch.equal(h, href)
                assert torch.equal((vr, vx)[over], (r, x)[over])
                assert torch.equal(y.codes, qref.codes) if quantize else torch.equal(y, ref)
                _clean((vx, bx), (vr, br))
