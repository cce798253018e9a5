"""How precisely the mixture-of-experts layer holds a hidden value between the
projections, seen through projections that pass single values on.

Token t is zero but for three values: gate and up take one product each from it,
so that a hidden value is the fp32 rounding of a product of two exact fp16 ones
(2^-24 of it) and is then held as fp16 plus 2^-11 times fp16.  The first is off by
at most half its last place, 2^-11 of the power of two below the value (2^-25 where
it is subnormal), and the second by 2^-12 of that, or 2^-36 in all: within
2^-22 of the value (2^-24 before, 2^-23 held, both at its larger end) plus 2^-36.
y is one or two such values times a power of two, summed in fp32, rounded to fp16.
"""
import pytest
import torch

import dense_tiled_gemm_fp16_gb300 as g

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


def stored(w, layout):
    """w [1, in, out] on the device, for each kernel of the layer: by TMA in either order,
    rows along the contracted axis or the other one that start anywhere, no unit stride."""
    if layout in ("nk", "odd rows"):
        w = w.transpose(1, 2)
    if layout in ("nk", "kn"):
        v = w.contiguous().to(DEV)
    elif layout == "every":
        v = torch.zeros(tuple(w.shape) + (2,), dtype=torch.float16, device=DEV)[..., 0]
        v.copy_(w)
    else:
        e, r, c = w.shape
        v = torch.zeros((e, r, c + 5), dtype=torch.float16, device=DEV)[:, :, 3:c + 3]
        v.copy_(w)
    return v.transpose(1, 2) if layout in ("nk", "odd rows") else v


LAYOUTS = ["nk", "kn", "odd rows", "odd columns", "every"]


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("T", [1, 5, 20, 50])
def test_hidden_values_of_every_size(T, layout):
    """Each output is one hidden value: 2^-24 to 2^14 in size, brought near 1 by powers of two."""
    F = D = 128
    gen = torch.Generator().manual_seed(T)
    e = torch.randint(-12, 8, (F,), generator=gen)
    gate, up, down = (torch.zeros((1, D, F)).half() for _ in range(3))
    gate[0, 0] = ((1 + torch.rand(F, generator=gen)) * torch.exp2(e.float())).half()
    up[0, 1] = ((1 + torch.rand(F, generator=gen)) * torch.exp2((e - 1).float())).half()
    x = torch.zeros((T, D)).half()
    x[:, 0] = (0.5 + 0.5 * torch.rand(T, generator=gen)).half()
    x[:, 1] = (0.5 + 0.5 * torch.rand(T, generator=gen)).half()
    s = torch.exp2(torch.clamp(-2.0 * e, -14, 15))
    down[0] = torch.diag(s).half()
    y, _, _ = g.moe_few(x.to(DEV), torch.zeros((D, 1), dtype=torch.float16, device=DEV),
                        *(stored(w, layout) for w in (gate, up, down)), 1, act="none")
    h = (x[:, :1].double() * gate[0, 0].double()) * (x[:, 1:2].double() * up[0, 1].double())
    ref, off = h * s.double(), s.double() * (2.0 ** -22 * h.abs() + 2.0 ** -36)
    tol = off + 2.0 ** -11 * (ref.abs() + off) + 2.0 ** -25
    err = (y.cpu().double() - ref).abs()
    assert (err <= tol).all(), float((err / tol).max())


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("size", [2.0 ** -11, 2.0 ** -4, 1.0, 2.0 ** 6])
def test_differences_of_hidden_values(size, layout):
    """Outputs are the differences of neighbouring hidden values that agree to 9 bits or more:
    a second half that were lost, or counted at another size, would be all that is left."""
    T, D, F = 9, 128, 256
    gen = torch.Generator().manual_seed(int(size * 4096))
    gate, up, down = torch.zeros((1, D, F)).half(), torch.zeros((1, D, F)).half(), torch.zeros((1, F, D)).half()
    a = ((1 + torch.rand(D, generator=gen)) * size).half()
    b = ((1 + torch.rand(D, generator=gen)) * size).half()
    gate[0, 0, 0::2] = gate[0, 0, 1::2] = a
    up[0, 1, 0::2] = b
    up[0, 1, 1::2] = (b.view(torch.int16) + 1).view(torch.float16)   # the next larger one
    x = torch.zeros((T, D)).half()
    x[:, :2] = (0.5 + 0.5 * torch.rand((T, 2), generator=gen)).half()
    s = 1.0 if size > 1 else 64.0
    i = torch.arange(D)
    down[0, 2 * i + 1, i], down[0, 2 * i, i] = s, -s
    y, _, _ = g.moe_few(x.to(DEV), torch.zeros((D, 1), dtype=torch.float16, device=DEV),
                        *(stored(w, layout) for w in (gate, up, down)), 1, act="none")
    h = (x[:, :1].double() * gate[0, 0].double()) * (x[:, 1:2].double() * up[0, 1].double())
    ref = s * (h[:, 1::2] - h[:, 0::2])
    off = s * 2 * (2.0 ** -22 * h[:, 1::2].abs() + 2.0 ** -36)
    tol = off + 2.0 ** -11 * (ref.abs() + off) + 2.0 ** -25
    err = (y.cpu().double() - ref).abs()
    assert (err <= tol).all(), float((err / tol).max())
    if size >= 2.0 ** -4:   # (smaller ones' differences are under fp16's smallest step)
        assert bool((ref.abs() > 4 * tol).any())


@pytest.mark.parametrize("layout", LAYOUTS)
def test_small_tokens(layout):
    """Tokens of deviation 2^-8: hidden values near 2^-17, outputs near 2^-12.  One rounding to
    fp16 leaves 2^-12 of an output's norm or so (a uniform error of half a last place: at most
    2^-11 / sqrt 3); nothing else may show."""
    T, D, F = 4, 1024, 1024
    gen = torch.Generator().manual_seed(7)
    x = (torch.randn((T, D), generator=gen) * 2.0 ** -8).half()
    gate, up = ((torch.randn((1, D, F), generator=gen) * D ** -0.5).half() for _ in range(2))
    down = torch.randn((1, F, D), generator=gen).half()
    y, _, _ = g.moe_few(x.to(DEV), torch.zeros((D, 1), dtype=torch.float16, device=DEV),
                        *(stored(w, layout) for w in (gate, up, down)), 1)
    h = torch.nn.functional.silu(x.double() @ gate[0].double()) * (x.double() @ up[0].double())
    ref = h @ down[0].double()
    rel = ((y.cpu().double() - ref).norm() / ref.norm()).item()
    assert rel <= 2.0 ** -11 / 3 ** 0.5 * 1.5, rel
