"""Calls of the 8-bit operators that their documentation allows and that are made less often: 16-bit rows at any
strides, matrices of two arrays, batches back to 16 bits, the most groups, workspaces used again.
"""
import pytest
import torch

import dense_tiled_gemm_fp16_gb300 as g
from tests.test_fp8_gpu import _near, _values

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
TYPES = [torch.float16, torch.bfloat16]


@pytest.fixture(autouse=True)
def _clean():
    yield
    g.gemm_f16_set_option(g.OPT_PAIR, 0)
    assert g.gemm_f16_device_status() == 0


def _normal(*shape, seed, dtype, scale=1.0):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    return torch.empty(shape, dtype=dtype, device=DEV).normal_(0.0, scale, generator=gen)


def _views(x):
    """x at strides of its own: transposed, rows and values apart, rows that start anywhere."""
    m, k = x.shape
    wide = torch.zeros((2 * m, 3 * k + 1), dtype=x.dtype, device=DEV)
    wide[::2, 1::3] = x
    off = torch.zeros((m, k + 3), dtype=x.dtype, device=DEV)
    off[:, 3:] = x
    return x.t().contiguous().t(), wide[::2, 1::3], off[:, 3:]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,N,K", [(1, 200, 300), (16, 512, 4200), (70, 60, 513), (500, 700, 1000)])
@pytest.mark.parametrize("form", [1, 2])
def test_products_of_16_bit_rows_at_any_strides(M, N, K, dtype, form):
    g.gemm_f16_set_option(g.OPT_PAIR, form)
    x, b = _normal(M, K, seed=1, dtype=dtype), g.fp8_quantize(_normal(N, K, seed=2, dtype=dtype))
    ref = g.fp8_mm(g.fp8_quantize(x), b, dtype=dtype)
    for v in _views(x):
        assert torch.equal(g.fp8_mm(v, b, dtype=dtype), ref)


@pytest.mark.parametrize("dtype", TYPES)
def test_grouped_products_of_16_bit_rows_at_any_strides(dtype):
    x, b = _normal(300, 520, seed=1, dtype=dtype), g.fp8_quantize(_normal(4, 300, 520, seed=2, dtype=dtype))
    counts = torch.tensor([100, 0, 150, 50], dtype=torch.int32, device=DEV)
    ref = g.fp8_grouped_mm(g.fp8_quantize(x), b, counts, dtype=dtype)
    for v in _views(x):
        assert torch.equal(g.fp8_grouped_mm(v, b, counts, dtype=dtype), ref)


def test_matrices_of_two_arrays():
    """Codes and scales that the caller keeps apart, as the C functions take them."""
    x, w = _normal(90, 700, seed=1, dtype=torch.float16), _normal(3, 200, 700, seed=2, dtype=torch.float16)
    two = lambda q: g.Fp8Matrix(q.codes.clone(), q.scales.clone(), q.rows, q.k, q.batch)  # noqa: E731
    a, b = g.fp8_quantize(x), g.fp8_quantize(w)
    one = g.fp8_quantize(w[1])
    counts = torch.tensor([30, 20, 40], dtype=torch.int32, device=DEV)
    assert torch.equal(g.fp8_mm(two(a), two(one)), g.fp8_mm(a, one))
    assert torch.equal(g.fp8_grouped_mm(two(a), two(b), counts, act="silu", b_up=two(b)),
                       g.fp8_grouped_mm(a, b, counts, act="silu", b_up=b))
    assert torch.equal(g.fp8_dequantize(two(b)), g.fp8_dequantize(b))


@pytest.mark.parametrize("to", TYPES + [torch.float32])
@pytest.mark.parametrize("batch,rows,k", [(1, 3, 40), (5, 130, 513), (7, 33, 1024), (300, 2, 7)])
def test_batches_back(batch, rows, k, to):
    x = _values((batch, rows, k), batch + k, torch.bfloat16).to(DEV)
    y = g.fp8_dequantize(g.fp8_quantize(x), dtype=to)
    assert y.shape == x.shape
    assert torch.equal(y, torch.stack([g.fp8_dequantize(g.fp8_quantize(v), dtype=to) for v in x]))


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("kind", ["one each", "one has all", "the last has all", "uneven"])
def test_the_most_groups(kind, gated):
    G, N, K, R = fp8_groups(), 130, 200, 700
    counts = torch.zeros(G, dtype=torch.int32)
    if kind == "one each":
        counts[:] = 1
    elif kind == "one has all":
        counts[77] = R
    elif kind == "the last has all":
        counts[-1] = R
    else:
        gen = torch.Generator().manual_seed(3)
        counts += torch.bincount(torch.randint(0, G, (R,), generator=gen) ** 2 // G, minlength=G).int()
    x = _normal(R, K, seed=1, dtype=torch.float16)
    ws = [g.fp8_quantize(_normal(G, N, K, seed=2 + i, dtype=torch.float16)) for i in range(1 + gated)]
    out = torch.full((R, N), -7.0, dtype=torch.float16, device=DEV)
    g.fp8_grouped_mm(x, ws[0], counts.to(DEV), act="silu" if gated else "none", b_up=ws[1] if gated else None, out=out)
    used = int(counts.sum())
    assert (out[used:] == -7.0).all()
    a = g.fp8_dequantize(g.fp8_quantize(x[:used]), dtype=torch.float32).double()
    which = torch.repeat_interleave(torch.arange(G), counts.long()).to(DEV)
    sums, sizes = [], []
    for w in ws:
        b = g.fp8_dequantize(w, dtype=torch.float32).double()
        v, s = torch.empty((used, N), dtype=torch.float64, device=DEV), torch.empty((used, N), dtype=torch.float64, device=DEV)
        for i in which.unique().tolist():
            at = which == i
            v[at], s[at] = a[at] @ b[i].T, a[at].abs() @ b[i].abs().T
        sums.append(v.cpu().numpy()), sizes.append(s.cpu().numpy())
    _near(out[:used], sums, sizes, K, "silu" if gated else "none")


def fp8_groups():
    from dense_tiled_gemm_fp16_gb300 import fp8
    return fp8.MAX_GROUPS


def test_a_workspace_used_again_at_once():
    """Calls one after the other quantise into the memory that the one before has let go: each reads its own."""
    b = g.fp8_quantize(_normal(300, 1000, seed=1, dtype=torch.float16))
    xs = [_normal(m, 1000, seed=m, dtype=torch.float16) for m in (16, 600, 40, 16, 3000, 16, 600)]
    refs = [g.fp8_mm(g.fp8_quantize(x), b) for x in xs]
    torch.cuda.synchronize()
    for _ in range(20):
        outs = [g.fp8_mm(x, b) for x in xs]
        assert all(torch.equal(o, r) for o, r in zip(outs, refs))
