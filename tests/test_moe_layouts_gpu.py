"""The expert layer's weights as callers may hold them: lengths that no vector divides, starts one value
off, orders that differ from one projection to the next, experts that interleave, overlap or are one and the
same; few tokens and many for each, so that every form of both experts' kernels runs.

Values are held to check()'s tolerances (tests/test_moe_gpu.py); weights at strides that TMA
can address are also compared bit for bit with a contiguous copy of the same values.
"""
import pytest
import torch

import dense_tiled_gemm_fp16_gb300 as g
from tests.test_moe_gpu import check, make, stored

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


def off_by(w, lead, layout):
    """w on the device, its first value `lead` elements past an aligned place, rows as long as they are
    ('odd nk', 'odd kn'), or with every element two apart ('odd every')."""
    v = w.transpose(1, 2) if layout == "odd nk" else w
    step = 2 if layout == "odd every" else 1
    flat = torch.full((lead + v.numel() * step + 7,), float("nan"), dtype=torch.float16, device=DEV)
    e, r, c = v.shape
    out = flat.as_strided((e, r, c), (r * c * step, c * step, step), lead)
    out.copy_(v)
    return out.transpose(1, 2) if layout == "odd nk" else out


# 8 tokens and fewer, to 16, to 32, more; odd sizes throughout, experts with several pieces of 8 and 16 tokens
SHAPES = [(1, 31, 17, 3, 2), (5, 1023, 77, 6, 3), (8, 129, 515, 2, 2), (9, 257, 129, 6, 3), (16, 257, 131, 6, 3),
          (20, 1001, 67, 2, 1), (32, 70, 33, 9, 4), (33, 131, 70, 9, 4), (40, 37, 1023, 4, 2), (64, 515, 203, 8, 8),
          (64, 203, 77, 2, 1), (64, 65, 31, 512, 8)]


@pytest.mark.parametrize("layout", ["odd nk", "odd kn", "odd every"])
@pytest.mark.parametrize("T,D,F,E,top", SHAPES)
def test_odd_lengths(T, D, F, E, top, layout):
    x, router, gate, up, down = make(T, D, F, E, T + D + F)
    ws = [off_by(w, lead, layout) for w, lead in ((gate, 0), (up, 3), (down, 5))]
    renorm, act = T % 2 == 0, ("silu", "gelu", "relu")[T % 3]
    args = (x.to(DEV), router.to(DEV), *ws, top)
    got = g.moe_few(*args, act=act, renormalize=renorm)
    check(x, router, gate, up, down, top, act, renorm, got)
    assert all(torch.equal(a, b) for a, b in zip(got, g.moe_few(*args, act=act, renormalize=renorm)))
    assert g.gemm_f16_device_status() == 0


@pytest.mark.parametrize("layout", ["odd nk", "odd kn", "odd every"])
@pytest.mark.parametrize("T", [2, 12, 24, 48])
def test_whole_lengths_that_start_one_value_off(T, layout):
    x, router, gate, up, down = make(T, 320, 192, 5, T)
    ws = [off_by(w, 1, layout) for w in (gate, up, down)]
    got = g.moe_few(x.to(DEV), router.to(DEV), *ws, 3)
    check(x, router, gate, up, down, 3, "silu", True, got)


@pytest.mark.parametrize("orders", ["nk nk kn", "kn kn nk", "nk kn nk", "kn nk kn", "nk nk odd"])
@pytest.mark.parametrize("T", [1, 13, 40])
def test_orders_that_differ(T, orders):
    x, router, gate, up, down = make(T, 264, 136, 7, T)
    ws = [off_by(w, 3, "odd kn") if o == "odd" else stored(w, o) for w, o in zip((gate, up, down), orders.split())]
    got = g.moe_few(x.to(DEV), router.to(DEV), *ws, 2)
    check(x, router, gate, up, down, 2, "silu", True, got)


def _views(name, base, flat):
    """The three projections of 6 experts of 128 x 64 at strides of that name."""
    shapes = [tuple(w.shape) for w in base]
    if name == "interleaved kn":
        return [w.transpose(0, 1).contiguous().transpose(0, 1) for w in base]
    if name == "interleaved nk":
        return [w.permute(2, 0, 1).contiguous().permute(1, 2, 0) for w in base]
    if name == "shared":
        return [w[:1].expand(6, *w.shape[1:]) for w in base]
    strides = {"overlapping rows kn": lambda r, c: (r * c, 8, 1), "overlapping rows nk": lambda r, c: (r * c, 1, 8),
               "experts 8 values apart": lambda r, c: (8, 1, r)}[name]
    return [flat.as_strided(s, strides(*s[1:])) for s in shapes]


@pytest.mark.parametrize("T", [3, 40])
@pytest.mark.parametrize("name", ["interleaved kn", "interleaved nk", "overlapping rows kn", "overlapping rows nk",
                                  "experts 8 values apart", "shared"])
def test_strides_that_overlap_or_interleave(T, name):
    x, router, gate, up, down = make(T, 128, 64, 6, T)
    base = [w.to(DEV) for w in (gate, up, down)]
    flat = torch.cat([w.flatten() for w in base])
    ws = _views(name, base, flat)
    got = g.moe_few(x.to(DEV), router.to(DEV), *ws, 3)
    check(x, router, *(w.cpu() for w in ws), 3, "silu", True, got)
    if name != "shared":   # (a stride of 0 is read by another kernel, which sums in another order)
        same = g.moe_few(x.to(DEV), router.to(DEV), *(stored(w.cpu(), "nk" if w.stride(1) == 1 else "kn") for w in ws), 3)
        assert all(torch.equal(a, b) for a, b in zip(got, same))
