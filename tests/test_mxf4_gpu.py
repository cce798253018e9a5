"""MXFP4 quantisation, its inverse and the product against a 64-bit restatement.

The conversions have one right answer, so they are compared bit for bit.  The
product of two quantised matrices sums exact terms in fp32: with inputs whose
sums are exact too (small integers) it is compared bit for bit, otherwise to
fp32 accumulation plus one rounding to fp16, |d| <= 2^-11 |c| + 2^-24 (the
store's rounding, half an ulp) + 2^-22 sum_k |a_k b_k| (an fp32 sum that loses
at most two bits below its largest term at each of its joins).
"""
import numpy as np
import pytest
import torch

import dense_tiled_gemm_fp16_gb300 as g
from tests.mxf4_reference import dequantize64, quantize64, scales_plain

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def _x(shape, dtype, seed, spread=True):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=gen)
    if spread:   # block maxima over many powers of two
        x = x * torch.exp2(torch.randint(-12, 9, shape[:-1] + (1,), generator=gen).float())
    return x.to(dtype)


def _check_quantized(x, q, rows, k):
    """codes and scales of one matrix against the restatement, padding included."""
    ref_codes, ref_scales = quantize64(x)
    nb = -(-k // 32)
    codes = q.codes.cpu().numpy().reshape(rows, nb * 16)
    lo, hi = codes & 15, codes >> 4
    got = np.stack([lo, hi], -1).reshape(rows, nb * 32)
    scales = scales_plain(q.scales.cpu().numpy(), rows, k)
    assert np.array_equal(scales, ref_scales)
    # a zero may carry either sign
    same = (got == ref_codes) | (((got & 7) == 0) & ((ref_codes & 7) == 0))
    assert same.all(), np.argwhere(~same)[:5]
    assert not got[:, k:].any()


@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("rows,k", [(1, 1), (1, 32), (1, 33), (3, 31), (16, 256), (127, 257), (128, 128), (129, 100),
                                    (5, 1000), (300, 8), (257, 4097)])
@pytest.mark.parametrize("layout", ["rows", "transposed", "pitched"])
def test_quantize(rows, k, dtype, layout):
    dt = DTYPES[dtype]
    x = _x((rows, k), dt, rows * 1000 + k)
    if layout == "transposed":
        d = x.t().contiguous().to(DEV).t()
    elif layout == "pitched":   # an odd pitch and an odd start: no 16-byte alignment
        buf = torch.zeros((rows, k + 3), dtype=dt, device=DEV)
        buf[:, 1:k + 1] = x.to(DEV)
        d = buf[:, 1:k + 1]
    else:
        d = x.to(DEV)
    q = g.mxf4_quantize(d)
    _check_quantized(x.double().numpy(), q, rows, k)
    ref = dequantize64(*quantize64(x.double().numpy()))[:, :k]
    for out in DTYPES.values():
        y = g.mxf4_dequantize(q, out)
        assert torch.equal(y.cpu().double(), torch.from_numpy(ref).to(out).double())


@pytest.mark.parametrize("dtype", sorted(DTYPES))
def test_quantize_rounds_ties_and_edges(dtype):
    """Every midpoint, both signs, at several scales; zeros; the type's ends."""
    mids = [0.0, 0.25, 0.5, 0.75, 1.0, 1.25, 1.5, 1.75, 2.0, 2.5, 3.0, 3.5, 4.0, 5.0, 6.0, 7.0, 7.5]
    row = torch.tensor(mids[:15] + [-v for v in mids[:15]] + [4.0, 7.0])
    rows = [row * s for s in (1.0, 0.25, 16.0)]
    rows += [torch.zeros(32), torch.full((32,), 7.75), torch.cat([torch.zeros(31), torch.tensor([-1e-4])])]
    fin = torch.finfo(DTYPES[dtype])
    for edge in (fin.max, fin.tiny, fin.smallest_normal * fin.eps):   # largest, smallest normal, smallest subnormal
        rows.append(torch.cat([torch.tensor([edge, -edge, edge / 2, 0.0]), torch.zeros(28)]))
    x = torch.stack(rows).to(DTYPES[dtype])
    q = g.mxf4_quantize(x.to(DEV))
    _check_quantized(x.double().numpy(), q, x.shape[0], 32)
    ref = dequantize64(*quantize64(x.double().numpy()))
    assert np.array_equal(g.mxf4_dequantize(q, torch.float32).cpu().double().numpy(), ref)


@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_a_block_with_no_finite_maximum_is_nan(dtype, bad):
    x = _x((130, 96), DTYPES[dtype], 7)
    x[129, 40] = bad
    for d in (x.to(DEV), x.t().contiguous().to(DEV).t()):
        y = g.mxf4_dequantize(g.mxf4_quantize(d), torch.float32).cpu()
        assert torch.isnan(y[129, 32:64]).all()
        y[129, 32:64] = 0
        assert torch.isfinite(y).all()


def test_batches_and_axes():
    x = _x((5, 70, 130), torch.float16, 3)
    d = x.to(DEV)
    q = g.mxf4_quantize(d)
    t = g.mxf4_quantize(d.transpose(1, 2).contiguous(), axis=-2)
    assert q.shape == t.shape == (5, 70, 130) and torch.equal(q.codes, t.codes) and torch.equal(q.scales, t.scales)
    y = g.mxf4_dequantize(q)
    for b in range(5):
        one = g.mxf4_quantize(d[b])
        assert torch.equal(g.mxf4_dequantize(one), y[b])
    shared = g.mxf4_dequantize(g.mxf4_quantize(d[:1].expand(3, 70, 130)))
    assert torch.equal(shared, y[:1].expand(3, 70, 130))


def _mm_check(a, b, c, bias=None, act="none"):
    """a [M, K], b [N, K]: 64-bit values of the quantised operands."""
    v, size = a @ b.T, np.abs(a) @ np.abs(b).T
    slope = 1.0
    if bias is not None:
        v, size = v + bias, size + np.abs(bias)
    if act == "relu":
        v = np.maximum(v, 0)
    elif act in ("silu", "gelu"):
        t = torch.from_numpy(v)
        v = getattr(torch.nn.functional, act)(t).numpy()
        slope = 1.13   # the largest slope of either
    tol = 2.0 ** -11 * np.abs(v) + 2.0 ** -24 + slope * 2.0 ** -22 * size + 2.0 ** -20 * np.abs(v)
    err = np.abs(c.astype(np.float64) - v)
    assert np.isfinite(c).all() and (err <= tol).all(), (err / tol).max()


def _operands(M, N, K, seed):
    x = _x((M, K), torch.float16, seed, spread=False)
    w = _x((N, K), torch.float16, seed + 1, spread=False) * K ** -0.5
    return x.to(DEV), w.half().to(DEV)


SHAPES = [(1, 1, 1), (1, 7, 31), (1, 128, 64), (1, 2048, 7168), (2, 130, 96), (16, 300, 1000), (17, 257, 512),
          (33, 129, 4097), (64, 65, 256), (65, 64, 320), (130, 70, 65), (128, 128, 4160), (200, 33, 2048),
          (300, 513, 1100), (1000, 600, 200), (129, 2, 8192), (515, 1030, 2500)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_mm_of_integers_is_exact(M, N, K):
    """e2m1 holds -4 .. 4 and 6 whole under the scale 1 that a maximum of 4 to 6
    gives: integer operands pass unchanged and every sum below 2^11 is exact."""
    rng = np.random.default_rng(M * 7 + N * 3 + K)
    a = rng.integers(-1, 2, (M, K)).astype(np.float16)
    b = rng.integers(-1, 2, (N, K)).astype(np.float16)
    a[:, ::32], b[:, ::32] = 4, 0   # the first value of each block sets its scale and adds nothing
    A, B = torch.from_numpy(a).to(DEV), torch.from_numpy(b).to(DEV)
    c = g.mxf4_mm(A, g.mxf4_quantize(B)).cpu().numpy().astype(np.float64)
    ref = a.astype(np.float64) @ b.astype(np.float64).T
    assert np.abs(ref).max() <= 2048 and np.array_equal(c, ref)


@pytest.mark.parametrize("M,N,K", SHAPES + [(1500, 1300, 700), (4100, 520, 384)])
def test_mm(M, N, K):
    x, w = _operands(M, N, K, M + N + K)
    qa, qb = g.mxf4_quantize(x), g.mxf4_quantize(w)
    a, b = (dequantize64(*quantize64(t.cpu().double().numpy()))[:, :K] for t in (x, w))
    c = g.mxf4_mm(qa, qb)
    _mm_check(a, b, c.cpu().numpy())
    assert torch.equal(c, g.mxf4_mm(x, qb))
    assert g.gemm_f16_device_status() == 0


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
@pytest.mark.parametrize("M,N,K", [(5, 200, 320), (150, 75, 640), (700, 900, 256)])
def test_mm_bias_act_and_strided_out(M, N, K, act):
    x, w = _operands(M, N, K, 11)
    bias = _x((N,), torch.float16, 12, spread=False).to(DEV)
    buf = torch.full((M + 2, N + 5), -7.0, dtype=torch.float16, device=DEV)
    out = buf[1:M + 1, 3:N + 3]
    g.mxf4_mm(x, g.mxf4_quantize(w), bias=bias, act=act, out=out)
    a, b = (dequantize64(*quantize64(t.cpu().double().numpy()))[:, :K] for t in (x, w))
    _mm_check(a, b, out.cpu().numpy(), bias.cpu().double().numpy(), act)
    buf[1:M + 1, 3:N + 3] = -7.0
    assert (buf == -7.0).all()   # nothing around the output was written


def test_mm_scales_of_every_size_and_nan_blocks():
    """Scales at both ends of their range meet; a NaN block reaches its row and column alone."""
    K = 128
    a = torch.ones((4, K))
    a[1], a[2] = 2.0 ** -120, 2.0 ** 120
    a[3, 70] = float("nan")
    b = torch.ones((3, K))
    b[1], b[2] = 2.0 ** 118, 2.0 ** -116
    qa, qb = g.mxf4_quantize(a.to(DEV)), g.mxf4_quantize(b.to(DEV))
    c = g.mxf4_mm(qa, qb).cpu().double()
    ref = (a.double() @ b.double().T).to(torch.float16).double()   # 128 * 2^120 * 2^118 is infinite in fp32 too
    assert torch.isnan(c[3]).all()
    assert torch.equal(c[:3], ref[:3])


@pytest.mark.parametrize("M", [3, 300])
def test_stalled_wait_reports_timeout_and_the_context_survives(M):
    x, w = _operands(M, 260, 1024, 5)
    q = g.mxf4_quantize(w)
    ref = g.mxf4_mm(x, q)
    g.gemm_f16_device_status(reset=True)
    try:
        g.gemm_f16_set_option(g.OPT_TIMEOUT_MS, 50)
        g.gemm_f16_set_option(g.OPT_TEST_STALL, 1)
        g.mxf4_mm(x, q)
        assert g.gemm_f16_device_status(reset=True) == g.ERR_TIMEOUT
    finally:
        g.gemm_f16_set_option(g.OPT_TEST_STALL, 0)
        g.gemm_f16_set_option(g.OPT_TIMEOUT_MS, 0)
    assert torch.equal(g.mxf4_mm(x, q), ref) and g.gemm_f16_device_status() == 0


def test_another_stream_and_a_graph():
    x, w = _operands(20, 512, 2048, 9)
    q = g.mxf4_quantize(w)
    ref = g.mxf4_mm(x, q)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    c = g.mxf4_mm(x, q, stream=s)
    s.synchronize()
    assert torch.equal(c, ref)
    out = torch.empty_like(ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.mxf4_mm(x, q, out=out)
    x.mul_(-1)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, -ref)
