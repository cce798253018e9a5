"""The 8-bit products' rarer forms: weights of several bands, sums over a cluster of any size, scales at opposite ends.

The operands in 64 bits are what ``fp8_dequantize`` gives in fp32, which is exact; tolerances are those of the
other products (a sum over a cluster of c CTAs rounds K / (32 c) + c times, no more than K / 32 + 1 in order).
"""
import pytest
import torch

import dense_tiled_gemm_fp16_gb300 as g
from tests.test_fp8_gpu import _near

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(autouse=True)
def _clean():
    yield
    g.gemm_f16_set_option(g.OPT_PAIR, 0)
    assert g.gemm_f16_device_status() == 0


def _normal(*shape, seed, dtype, scale=1.0):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    return torch.empty(shape, dtype=dtype, device=DEV).normal_(0.0, scale, generator=gen)


def _held(q):
    return g.fp8_dequantize(q, dtype=torch.float32).double()


def _sums(a, b):
    """The product and the sums of its terms' magnitudes."""
    return (a @ b.T).cpu().numpy(), (a.abs() @ b.abs().T).cpu().numpy()


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("M,N,K", [(600, 4900, 8200), (1, 4352, 8192), (2000, 2600, 16400)])
def test_weights_of_several_bands(M, N, K, dtype):
    """More than 32 MB of weights: 15, 16 and 8 tiles of 256 in a band, the last one shorter."""
    g.gemm_f16_set_option(g.OPT_PAIR, 2)
    a = g.fp8_quantize(_normal(M, K, seed=1, dtype=dtype))
    b = g.fp8_quantize(_normal(N, K, seed=2, dtype=dtype, scale=K ** -0.5))
    v, size = _sums(_held(a), _held(b))
    _near(g.fp8_mm(a, b, dtype=dtype), [v], [size], K)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("counts", [(330, 0, 270), (1, 700, 40)])
def test_grouped_weights_of_several_bands(counts, gated):
    """15 tiles of 256 weight rows (with gate and up of 128) in a band, 20 and 39 in all."""
    N, K, rows = 4900, 8200, sum(counts)
    x = _normal(rows + 5, K, seed=3, dtype=F16)
    ws = [g.fp8_quantize(_normal(len(counts), N, K, seed=4 + i, dtype=F16, scale=K ** -0.5)) for i in range(1 + gated)]
    out = torch.full((rows + 5, N), -7.0, dtype=F16, device=DEV)
    g.fp8_grouped_mm(x, ws[0], torch.tensor(counts, dtype=torch.int32, device=DEV), act="silu" if gated else "none",
                     b_up=ws[1] if gated else None, out=out)
    assert (out[rows:] == -7.0).all()
    a, bs, at = _held(g.fp8_quantize(x)), [_held(w) for w in ws], 0
    for i, n in enumerate(counts):
        if n:
            both = [_sums(a[at:at + n], b[i]) for b in bs]
            _near(out[at:at + n], [v for v, _ in both], [s for _, s in both], K, "silu" if gated else "none")
        at += n


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("M,N,K", [
    (8, 512, 2100), (8, 512, 8200), (16, 700, 4200),            # columns of 16, clusters of 2, 8 and 4
    (32, 12800, 4200), (32, 512, 4200), (20, 300, 8200),        # of 32: 2, 4 and 8
    (64, 300, 8200), (40, 1000, 4200), (64, 10000, 4200),       # of 64: 8, 4 and 2
    (300, 48, 8200), (300, 64, 4200), (5000, 17, 4200),         # rows of C in the lanes, columns of 64 and 32
    (100, 100, 8200), (200, 200, 4200), (1200, 1100, 4200)])    # of 128: 8, 4 and 2
@pytest.mark.parametrize("bias,act", [(False, "none"), (True, "gelu"), (True, "silu")])
def test_sums_over_a_cluster(M, N, K, bias, act, dtype):
    g.gemm_f16_set_option(g.OPT_PAIR, 1)
    a = g.fp8_quantize(_normal(M, K, seed=1, dtype=dtype))
    b = g.fp8_quantize(_normal(N, K, seed=2, dtype=dtype, scale=K ** -0.5))
    t = _normal(N, seed=3, dtype=dtype) if bias else None
    v, size = _sums(_held(a), _held(b))
    if bias:
        extra = t.double().cpu().numpy()
        v, size = v + extra, size + abs(extra)
    for lead, pitch in ((0, 0), (3, 5)):   # and C's rows off 16 bytes
        ld = (N + 7) // 8 * 8 + lead + pitch
        buf = torch.full((M + 2, ld), -7.0, dtype=dtype, device=DEV)
        out = buf[1:M + 1, lead:lead + N]
        g.fp8_mm(a, b, bias=t, act=act, out=out)
        _near(out, [v], [size], K, act)
        out.fill_(-7.0)
        assert (buf == -7.0).all()


@pytest.mark.parametrize("form", [1, 2])
@pytest.mark.parametrize("power", [0, 60, 100, 110])
def test_scales_at_opposite_ends(power, form):
    """Values of 2^power times values of 2^-power: the scales' product is near one, whatever either is."""
    M, N, K = 40, 300, 640
    g.gemm_f16_set_option(g.OPT_PAIR, form)
    for sign in (1, -1):
        x = _normal(M, K, seed=1, dtype=torch.float32).mul_(2.0 ** (sign * power))
        w = _normal(N, K, seed=2, dtype=torch.float32).mul_(2.0 ** (-sign * power))
        a, b = g.fp8_quantize(x), g.fp8_quantize(w)
        v, size = _sums(_held(a), _held(b))
        _near(g.fp8_mm(a, b, dtype=BF16), [v], [size], K)
