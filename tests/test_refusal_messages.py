"""A refused tensor is named in the terms of the call that refuses it (on the CPU)."""
import pytest
import torch

import dense_tiled_gemm_fp16_gb300 as g

H = torch.float16


def z(*s, dtype=H):
    return torch.zeros(s, dtype=dtype)


@pytest.mark.parametrize("which", ["x", "router", "out"])
def test_layer(which):
    a = dict(x=z(3, 16), router=z(16, 4), out=z(3, 16))
    a[which] = a[which].float()
    gate, down = z(4, 16, 8), z(4, 8, 16)
    with pytest.raises(TypeError, match=f"moe_few takes {which} "):
        g.moe_few(a["x"], a["router"], gate, gate, down, 2, out=a["out"])


def test_product():
    q = g.Mxf4Matrix(z(4 * 32, dtype=torch.uint8), z(512, dtype=torch.uint8), 4, 64)
    with pytest.raises(TypeError, match="mxf4_mm takes a "):
        g.mxf4_mm(z(3, 64, dtype=torch.float32), q)


def test_inverse_of_a_host_matrix():
    q = g.Mxf4Matrix(z(4 * 32, dtype=torch.uint8), z(512, dtype=torch.uint8), 4, 64)
    with pytest.raises(ValueError, match="CUDA device"):
        g.mxf4_dequantize(q)


@pytest.mark.gpu
@pytest.mark.parametrize("which", ["bias", "out"])
def test_product_on_the_device(which):
    w = torch.ones((4, 64), dtype=H, device="cuda:0")
    bad = {"bias": torch.zeros(4, device="cuda:0"), "out": torch.zeros((3, 4), device="cuda:0")}[which]
    with pytest.raises(TypeError, match=f"mxf4_mm takes {which} "):
        g.mxf4_mm(w[:3], g.mxf4_quantize(w), **{which: bad})
