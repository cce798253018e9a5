"""The weights' gradient where its rounding adds up most: rows of one sign.

A block of 128 threads takes 1024 values of a row at a time, eight a lane, each product added with one rounding:
8 ceil(d / 1024) of them in sequence, then five by the warp's tree and three over the four warps.  Every partial
sum is no more than the whole, so that dweights is within (8 ceil(d / 1024) + 8) 2^-24 of itself.
"""
import pytest
import torch

import dense_tiled_gemm_fp16_gb300 as g

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("top", [1, 2, 4, 8, 11])
@pytest.mark.parametrize("d", [1, 1023, 4100, 7168, 32768, 100001])
def test_dot_products_of_one_sign(d, top, dtype):
    T, E = 9, 5
    gen = torch.Generator().manual_seed(d + top)
    o = g.moe_sort(torch.randint(0, E, (T, top), generator=gen).int().to(DEV), E)
    dout = (torch.rand((T, d), generator=gen) + 0.5).to(dtype).to(DEV)
    y = (torch.rand((T * top, d), generator=gen) + 0.5).to(dtype).to(DEV)
    w = torch.rand((T, top), generator=gen).to(DEV)
    _, dw = g.moe_combine_grad(dout, y, o, w)
    v = (y[o.rows.long()].double() * dout.double()[:, None]).sum(dim=2)
    roundings = 8 * -(-d // 1024) + 8
    assert ((dw.double() - v).abs() <= roundings * 2.0 ** -24 * (1 + 2.0 ** -10) * v).all()
