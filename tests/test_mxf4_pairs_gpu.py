"""MXFP4 products by the CTA-pair kernel and of few columns: both tile widths, outputs
that TMA can store and outputs that it cannot, bias and activation far into
their tails, launch options.

Tolerances: a fp32 sum is off by at most 2^-22 of the sum of its terms'
magnitudes, an activation adds its slope (at most 1.13) of that and 2^-18 of its
own value, and the result is rounded to fp16 once (2^-11 of it, 2^-25 where it
is subnormal).
"""
import numpy as np
import pytest
import torch

import dense_tiled_gemm_fp16_gb300 as g
from tests.mxf4_reference import dequantize64, quantize64

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
# tiles of 256 x 256 for fewer turns, then of 256 x 128; more than one turn of either
SHAPES = [(1500, 2003, 300), (3001, 1999, 130), (3001, 2000, 97), (5000, 2049, 70)]


def _operands(M, N, K, seed, scale):
    gen = torch.Generator().manual_seed(seed)
    x = (torch.randn((M, K), generator=gen) * scale).half()
    w = (torch.randn((N, K), generator=gen) * K ** -0.5).half()
    return x, w


def _held(x):
    return dequantize64(*quantize64(x.double().numpy()))[:, :x.shape[1]]


def _check(a, b, bias, act, c):
    v, size = a @ b.T + bias, np.abs(a) @ np.abs(b).T + np.abs(bias)
    tol = 2.0 ** -22 * size
    if act == "relu":
        v = np.maximum(v, 0)
    elif act in ("silu", "gelu"):
        v = getattr(torch.nn.functional, act)(torch.from_numpy(v)).numpy()
        tol = 1.13 * tol + 2.0 ** -18 * np.abs(v)
    tol += 2.0 ** -11 * np.abs(v) + 2.0 ** -25
    err = np.abs(c.cpu().numpy().astype(np.float64) - v)
    assert (err <= tol).all(), (err / tol).max()


@pytest.mark.parametrize("act,scale", [("none", 1), ("relu", 1), ("silu", 8), ("gelu", 2.5)])
@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("lead,pitch", [(0, 8), (3, 5)])
def test_bias_activation_and_the_output_s_place(M, N, K, act, scale, lead, pitch):
    x, w = _operands(M, N, K, M + N + K, scale)
    bias = torch.randn(N, generator=torch.Generator().manual_seed(3)).half()
    ld = (N + 7) // 8 * 8 + pitch
    buf = torch.full((M + 2, ld), -7.0, dtype=torch.float16, device=DEV)
    out = buf[1:M + 1, lead:lead + N]
    g.mxf4_mm(x.to(DEV), g.mxf4_quantize(w.to(DEV)), bias=bias.to(DEV), act=act, out=out)
    _check(_held(x), _held(w), bias.double().numpy(), act, out)
    out.fill_(-7.0)
    assert (buf == -7.0).all()   # nothing around the output was written
    assert g.gemm_f16_device_status() == 0


@pytest.mark.parametrize("M,N,K", [(96, 96, 10500), (70, 200, 12000), (300, 16, 8192), (1000, 40, 4096), (513, 3, 2100),
                                   (20000, 33, 300)])
def test_few_columns_and_long_sums(M, N, K):
    x, w = _operands(M, N, K, M + N + K, 1)
    bias = torch.randn(N, generator=torch.Generator().manual_seed(3)).half()
    buf = torch.full((M + 1, N + 3), -7.0, dtype=torch.float16, device=DEV)
    out = buf[:M, :N]
    g.mxf4_mm(x.to(DEV), g.mxf4_quantize(w.to(DEV)), bias=bias.to(DEV), act="silu", out=out)
    _check(_held(x), _held(w), bias.double().numpy(), "silu", out)
    out.fill_(-7.0)
    assert (buf == -7.0).all()


def test_activations_of_extreme_sums():
    """Sums of every size from 2^-30 to infinity, of both signs, and NaN."""
    M, N, K = 1500, 2000, 32
    a, b = torch.ones((M, K)), torch.zeros((N, K))
    e = torch.arange(N) % 60 - 30.0
    b[:, 0] = torch.exp2(e) * torch.where(torch.arange(N) % 7 < 3, -1.0, 1.0)
    b[5, 0], a[9, 3] = 2.0 ** 127, float("nan")
    a[11, 0] = 2.0 ** 6   # 2^6 * 2^127: an infinite sum
    qa, qb = g.mxf4_quantize(a.to(DEV)), g.mxf4_quantize(b.to(DEV))
    with np.errstate(all="ignore"):
        v = torch.from_numpy((_held(a) @ _held(b).T).astype(np.float32)).double()
    for act in ("relu", "silu", "gelu"):
        c = g.mxf4_mm(qa, qb, act=act).cpu().double()
        ref = getattr(torch.nn.functional, act)(v)
        assert torch.isnan(c[9]).all() or act == "relu"
        rows = [r for r in range(M) if r != 9]
        c, r = c[rows], ref[rows]
        big = r.abs() > 65519   # beyond fp16
        assert torch.equal(torch.isinf(c), big) and torch.equal(torch.sign(c[big]), torch.sign(r[big]))
        err = (c - r).abs()[~big]
        assert (err <= (2.0 ** -11 + 2.0 ** -18) * r[~big].abs() + 2.0 ** -25).all()


def test_options_streams_and_repeats():
    x, w = _operands(1500, 2003, 520, 4, 1)
    q, x = g.mxf4_quantize(w.to(DEV)), x.to(DEV)
    ref = g.mxf4_mm(x, q)
    try:
        g.gemm_f16_set_option(g.OPT_PDL, 1)
        assert torch.equal(g.mxf4_mm(x, q), ref)
        assert torch.equal(g.mxf4_mm(x[:3], q), g.mxf4_mm(g.mxf4_quantize(x[:3]), q))
    finally:
        g.gemm_f16_set_option(g.OPT_PDL, 0)
    torch.cuda.synchronize()
    s = [torch.cuda.Stream() for _ in range(3)]
    got = [[g.mxf4_mm(x, q, stream=t) for t in s] for _ in range(5)]
    torch.cuda.synchronize()
    assert all(torch.equal(c, ref) for row in got for c in row)


def test_rows_past_4_gib_of_output():
    """An output of more than 2^31 elements: the last rows are where they belong."""
    M, N, K = 1100000, 2048, 32
    w = torch.zeros((N, K), dtype=torch.float16, device=DEV)
    w[:, 0] = 1
    x = torch.zeros((M, K), dtype=torch.float16, device=DEV)
    x[:, 0] = (torch.arange(M, device=DEV) % 7 - 3).half()
    c = g.mxf4_mm(x, g.mxf4_quantize(w))
    for lo in (0, 524288, M - 4096):
        assert torch.equal(c[lo:lo + 4096], x[lo:lo + 4096, :1].expand(4096, N))
