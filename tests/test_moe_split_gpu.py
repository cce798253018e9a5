"""How MXFP4 columns hold a token's and a hidden value, seen one by one.

With one expert, no activation, gate and down that pass single values on and up that is 1, y is a
token's value held twice: among the tokens and among the hidden values.  The columns of a block of 32
leave at most 2^-21 of a unit 2^s whose triple is below the block's largest magnitude, so less than
2^-22.5 of that magnitude; the sums of a value's columns are exact in fp32 (24 bits from 2^(s + 2) down
to the last column's half unit, 2^(s - 21)).  So each output is within 2 * 2^-22.5 of its block's
largest magnitude, and half a last place of fp16, of the token's value.
"""
import pytest
import torch

import dense_tiled_gemm_fp16_gb300 as g
from tests.test_moe_gpu import held

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BLOCKS = 6


@pytest.mark.parametrize("T", [1, 3, 16, 40, 64])
# largest magnitudes of a block: powers of two, at and past the two ends of a unit's range, any
@pytest.mark.parametrize("top", [1.0, 1.25, 1.5, 1.5009765625, 1.75, 1.9990234375, None])
@pytest.mark.parametrize("spread", [0, 6, 10, 13])   # the other values: of the same size, 2^-6, 2^-10, 2^-13 of it
def test_columns_leave_less_than_they_say(T, top, spread):
    F = 32 * BLOCKS
    D = F + 32
    gen = torch.Generator().manual_seed(T + spread)
    size = torch.exp2(torch.randint(-8, 9, (T, BLOCKS, 1), generator=gen).float())
    v = (2 * torch.rand((T, BLOCKS, 32), generator=gen) - 1) * 2.0 ** -spread
    big = 1 + torch.rand((T, BLOCKS), generator=gen) if top is None else torch.full((T, BLOCKS), top)
    v[:, :, 5] = big * (1 - 2 * torch.randint(0, 2, (T, BLOCKS), generator=gen))
    x = torch.zeros((T, D)).half()
    x[:, :F] = (v * size).half().view(T, F)
    x[:, F] = 1
    eye = torch.eye(F).half()
    gate, up, down = torch.zeros((1, D, F)).half(), torch.zeros((1, D, F)).half(), torch.zeros((1, F, D)).half()
    gate[0, :F], up[0, F], down[0, :, :F] = eye, 1, eye
    y, _, _ = g.moe_few(x.to(DEV), torch.zeros((D, 1), dtype=torch.float16, device=DEV),
                        *(g.mxf4_quantize(w.to(DEV), axis=-2) for w in (gate, up, down)), 1, act="none")
    ref = x[:, :F].double().view(T, BLOCKS, 32)
    off = 2 * 2.0 ** -22.5 * ref.abs().amax(dim=2, keepdim=True)
    err = (y[:, :F].cpu().double().view(T, BLOCKS, 32) - ref).abs()
    tol = off + 2.0 ** -11 * (ref.abs() + off) + 2.0 ** -25
    assert (err <= tol).all(), float((err / tol).max())
    assert not y[:, F:].any()


@pytest.mark.parametrize("outlier", [100.0, 1000.0, 4000.0])
@pytest.mark.parametrize("T", [4, 40])
def test_values_beside_an_outlier(T, outlier):
    """One value of each block is far larger and has weights of zero, as a hidden state's outliers may:
    what the others give is as near as without it.  Rounding y to fp16 leaves at most 2^-11 / sqrt 3 of
    its norm; the columns (2^-22.5 of the outlier for values of size 1) are under that."""
    D, F = 256, 128
    gen = torch.Generator().manual_seed(T)
    x = torch.randn((T, D), generator=gen).half()
    x[:, 7::32] = outlier * (1 - 2 * torch.randint(0, 2, (T, D // 32), generator=gen)).half()
    gate, up, down = ((torch.randn((1, a, b), generator=gen) * a ** -0.5).half() for a, b in ((D, F), (D, F), (F, D)))
    gate[0, 7::32], up[0, 7::32] = 0, 0
    dev, vals = zip(*(held(w) for w in (gate, up, down)))
    y, _, _ = g.moe_few(x.to(DEV), torch.zeros((D, 1), dtype=torch.float16, device=DEV), *dev, 1)
    gate, up, down = (v[0].double() for v in vals)
    ref = (torch.nn.functional.silu(x.double() @ gate) * (x.double() @ up)) @ down
    rel = ((y.cpu().double() - ref).norm() / ref.norm()).item()
    assert rel <= 2.0 ** -11 / 3 ** 0.5 * 1.5, rel
