"""What an Mxf4Matrix may be made of, without a GPU: contiguous bytes of the right number, on one device.

Its base addresses are all that the kernels get, so that anything else would be read as other values.
"""
import pytest
import torch

import dense_tiled_gemm_fp16_gb300 as g

U8 = torch.uint8


def codes(n=4 * 32, dtype=U8):
    return torch.zeros(n, dtype=dtype)


def scales(n=512, dtype=U8):
    return torch.zeros(n, dtype=dtype)


def test_bytes_in_any_shape_are_taken():
    for c, s in ((codes(), scales()), (codes().view(4, 32), scales().view(1, 1, 32, 16)), (codes(256)[128:], scales())):
        q = g.Mxf4Matrix(c, s, 4, 64)
        assert q.shape == (4, 64) and q.codes_ptr == c.data_ptr() and q.scales_ptr == s.data_ptr()


@pytest.mark.parametrize("c,s", [
    (codes(256)[::2], scales()), (codes(), scales(1024)[::2]),                 # every other byte
    (codes().view(32, 4).t(), scales()), (codes(), scales().view(16, 32).t()),   # turned round
    (codes(1).expand(128), scales()), (codes(), scales(1).expand(512)),        # one byte for all
    (codes().view(4, 32), scales(64).expand(8, 64))])
def test_strided_arrays_are_refused(c, s):
    with pytest.raises(ValueError, match="contiguous"):
        g.Mxf4Matrix(c, s, 4, 64)


@pytest.mark.parametrize("dtype", [torch.int8, torch.int32, torch.float16, torch.float32, torch.bool])
def test_arrays_of_other_types_are_refused(dtype):
    with pytest.raises(TypeError, match="uint8"):
        g.Mxf4Matrix(codes(dtype=dtype), scales(), 4, 64)
    with pytest.raises(TypeError, match="uint8"):
        g.Mxf4Matrix(codes(), scales(dtype=dtype), 4, 64)


@pytest.mark.parametrize("rows,k,batch", [(5, 64, None), (4, 65, None), (4, 64, 2), (0, 64, None), (4, 0, None), (4, 64, 0),
                                          (-4, -64, None), (4, 64, -1)])
def test_other_sizes_are_refused(rows, k, batch):
    with pytest.raises(ValueError):
        g.Mxf4Matrix(codes(), scales(), rows, k, batch)


def test_sizes_below_one_are_refused_whatever_the_arrays_hold():
    none = torch.zeros(0, dtype=U8)
    for rows, k, batch in ((0, 64, None), (4, 0, None), (4, 64, 0)):
        with pytest.raises(ValueError):
            g.Mxf4Matrix(none, none, rows, k, batch)
