"""The expert order and the rows that follow it, against 64 bits.

Places and copies are exact.  A weighted sum of n rows in fp32 is off by at most (n + 1) 2^-24 of the sum of
its terms' magnitudes and is rounded once (2^-11 of it in fp16, 2^-25 where it is subnormal; 2^-8 in bf16);
a dot product of d values, 8 a lane at a time and then a tree, by (d / 256 + 16) 2^-24.
"""
import numpy as np
import pytest
import torch

import dense_tiled_gemm_fp16_gb300 as g
from tests.fp8_reference import held64

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
TYPES = [torch.float16, torch.bfloat16]
HALF = {torch.float16: (2.0 ** -11, 2.0 ** -25), torch.bfloat16: (2.0 ** -8, 0.0)}


def _ids(T, top, E, seed, none=0.0):
    gen = torch.Generator().manual_seed(seed)
    p = torch.rand(E, generator=gen) ** 3 + 1e-3
    ids = torch.multinomial(p, T * top, replacement=True, generator=gen).view(T, top).int()   # one expert twice, too
    out = torch.rand((T, top), generator=gen) < none
    ids[out] = torch.tensor([-1, E, -2**31, 2**31 - 1], dtype=torch.int32)[torch.randint(0, 4, (int(out.sum()),), generator=gen)]
    return ids


def _plain_order(ids, E):
    flat = ids.flatten().long().numpy()
    good = (flat >= 0) & (flat < E)
    order = np.argsort(np.where(good, flat, E), kind="stable")
    rows = np.empty(flat.size, np.int32)
    rows[order] = np.arange(flat.size)
    return (np.where(good, rows, -1).reshape(ids.shape), np.where(good[order], order, -1),
            np.bincount(flat[good], minlength=E))


def _sorted(ids, E):
    o = g.moe_sort(ids.to(DEV), E)
    for got, want in zip(o, _plain_order(ids, E)):
        assert got.dtype is torch.int32 and (got.cpu().numpy() == want).all()
    return o


@pytest.mark.parametrize("none", [0.0, 0.3, 1.0])
@pytest.mark.parametrize("T,top,E", [(1, 1, 1), (1, 8, 64), (16, 8, 64), (128, 8, 512), (512, 8, 7), (1000, 3, 31), (4096, 1, 1),
                                     (513, 8, 512), (16384, 8, 64), (50001, 2, 100), (20000, 32, 256)])
def test_order(T, top, E, none):
    _sorted(_ids(T, top, E, T + E, none), E)


def _matrix(rows, d, dtype, seed, lead=0, pitch=0):
    """A matrix inside a buffer of -7, and the buffer."""
    gen = torch.Generator().manual_seed(seed)
    buf = torch.full((rows + 2, d + lead + pitch), -7.0, dtype=dtype, device=DEV)
    v = buf[1:rows + 1, lead:lead + d]
    v.copy_(torch.randn((rows, d), generator=gen))
    return v, buf


CASES = [(1, 1, 4, 1), (3, 2, 5, 70), (16, 8, 64, 7168), (40, 8, 16, 1030), (300, 5, 9, 2048), (70, 12, 30, 2056), (5, 32, 40, 4100)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,top,E,d", CASES)
@pytest.mark.parametrize("none,lead,pitch", [(0.0, 0, 0), (0.3, 3, 5), (0.3, 8, 8)])
def test_gather_combine_and_gradients(T, top, E, d, none, lead, pitch, dtype):
    o = _sorted(_ids(T, top, E, T + d, none), E)
    n, half = T * top, HALF[dtype]
    rows = o.rows.cpu().numpy()
    at, used = np.where(rows < 0, 0, rows), (rows >= 0)[..., None]
    x, _ = _matrix(T, d, dtype, 1, lead, pitch)
    out, buf = _matrix(n, d, dtype, 2, lead, pitch)
    buf.fill_(-7.0)
    assert g.moe_gather(x, o, out=out) is out
    want = torch.full((n, d), -7.0, dtype=dtype)
    order = o.order.cpu().long()
    want[order >= 0] = x.cpu()[order[order >= 0] // top]
    assert torch.equal(out.cpu(), want)   # places of no choice keep what they held
    out.fill_(-7.0)
    assert (buf == -7.0).all()

    y, _ = _matrix(n, d, dtype, 3, lead, pitch)
    gen = torch.Generator().manual_seed(4)
    w = torch.randn((T, top), generator=gen)
    w[torch.rand((T, top), generator=gen) < 0.1] = 0
    terms = y.double().cpu().numpy()[at] * used
    for weights in (None, w):
        z = terms if weights is None else terms * weights.double().numpy()[..., None]
        back, buf = _matrix(T, d, dtype, 2, lead, pitch)
        g.moe_combine(y, o, None if weights is None else weights.to(DEV), out=back)
        v = z.sum(axis=1)
        tol = (top + 1) * 2.0 ** -24 * np.abs(z).sum(axis=1) * (1 + half[0]) + half[0] * np.abs(v) + half[1]
        assert (np.abs(back.double().cpu().numpy() - v) <= tol).all()
        back.fill_(-7.0)
        assert (buf == -7.0).all()

    dout, _ = _matrix(T, d, dtype, 5, lead, pitch)
    dy, buf = _matrix(n, d, dtype, 6, lead, pitch)
    buf.fill_(-7.0)
    _, dw = g.moe_combine_grad(dout, y, o, w.to(DEV), out=dy)
    do = dout.double().cpu().numpy()
    v = np.full((n, d), -7.0)
    v[rows[rows >= 0]] = (w.double().numpy()[..., None] * do[:, None, :])[rows >= 0]
    tol = half[0] * np.abs(v) * (1 + 2.0 ** -20) + half[1] + 2.0 ** -24 * np.abs(v)
    assert (np.abs(dy.double().cpu().numpy() - v) <= tol).all()
    products = terms * do[:, None, :]
    err = np.abs(dw.double().cpu().numpy() - products.sum(axis=2))
    assert (err <= (d / 256 + 16) * 2.0 ** -24 * np.abs(products).sum(axis=2)).all()
    assert (dw.cpu().numpy()[rows < 0] == 0).all()
    dy.fill_(-7.0)
    assert (buf == -7.0).all()


def test_gradients_by_differences():
    """<moe_combine(moe_gather(x)), dout> moves by the gradients' share when x, y or the weights move."""
    T, top, E, d = 12, 3, 5, 40
    o = _sorted(_ids(T, top, E, 7, 0.2), E)
    gen = torch.Generator().manual_seed(9)
    x, dx, dout = (torch.randint(-8, 9, (T, d), generator=gen).half().to(DEV) for _ in range(3))
    w, dw = (torch.randint(-4, 5, (T, top), generator=gen).float().to(DEV) for _ in range(2))

    def loss(x, w):   # whole numbers small enough for fp16: exact
        y = g.moe_gather(x, o, out=torch.zeros((T * top, d), dtype=torch.float16, device=DEV))
        return (g.moe_combine(y, o, w).double() * dout.double()).sum().item()

    y = g.moe_gather(x, o, out=torch.zeros((T * top, d), dtype=torch.float16, device=DEV))
    gy, gw = g.moe_combine_grad(dout, y, o, w, out=torch.zeros_like(y))
    gx = g.moe_combine(gy, o)   # the gather's gradient
    assert loss(x + dx, w) - loss(x, w) == (gx.double() * dx.double()).sum().item()
    assert loss(x, w + dw) - loss(x, w) == (gw.double() * dw.double()).sum().item()


@pytest.mark.parametrize("T,top,E,k", [(1, 1, 1, 1), (3, 2, 5, 70), (16, 8, 64, 7168), (130, 3, 9, 4100), (1000, 5, 30, 513)])
def test_gather_of_8_bit_rows(T, top, E, k):
    o = _sorted(_ids(T, top, E, T + k), E)
    x, _ = _matrix(T, k, torch.float16, 1)
    q = g.moe_gather(g.fp8_quantize(x), o)
    from tests.test_fp8_gpu import _arrays, _same
    _same(q, g.moe_gather(x, o))
    assert np.array_equal(g.fp8_dequantize(q, dtype=torch.float32).double().cpu().numpy(),
                          held64(x)[o.order.cpu().numpy() // top])
    assert _arrays(q)


def test_no_tokens():
    o = g.moe_sort(torch.empty((0, 4), dtype=torch.int32, device=DEV), 6)
    assert o.rows.shape == (0, 4) and (o.group_rows == 0).all()
    x = torch.empty((0, 32), dtype=torch.float16, device=DEV)
    w = torch.empty((0, 4), device=DEV)
    assert g.moe_gather(x, o).shape == g.moe_combine(x, o, w).shape == (0, 32)
    assert [v.shape for v in g.moe_combine_grad(x, x, o, w)] == [(0, 32), (0, 4)]


def test_places_that_no_order_holds_are_taken_as_none():
    rows = torch.tensor([[0, 99], [-5, 3]], dtype=torch.int32, device=DEV)
    o = g.MoeOrder(rows, None, None)
    x, _ = _matrix(2, 64, torch.float16, 1)
    out = torch.full((4, 64), -7.0, dtype=torch.float16, device=DEV)
    g.moe_gather(x, o, out=out)
    assert torch.equal(out[0], x[0]) and torch.equal(out[3], x[1]) and (out[1:3] == -7).all()
    assert torch.equal(g.moe_combine(out, o), x)


def test_a_layer_of_experts_in_8_bits():
    """Norm, routing, both grouped products and the way back as they are used together, on a side stream and
    in a graph, against the same steps in 64 bits."""
    T, top, E, D, F = 150, 3, 8, 384, 256
    gen = torch.Generator().manual_seed(11)
    x = torch.randn((T, D), generator=gen).half().to(DEV)
    r = torch.randn((T, D), generator=gen).half().to(DEV)
    nw = torch.ones(D, dtype=torch.float16, device=DEV)
    gate, up, down = ((torch.randn(s, generator=gen) * s[1] ** -0.5).half().to(DEV) for s in ((E, D, F), (E, D, F), (E, F, D)))
    qg, qu, qd = (g.fp8_quantize(v, axis=-2) for v in (gate, up, down))
    ids = _ids(T, top, E, 12, 0.1)
    w = torch.rand((T, top), generator=gen).to(DEV)
    dev_ids = ids.to(DEV)

    def layer():
        q, h = g.rms_norm(x, nw, residual=r, quantize=True)
        o = g.moe_sort(dev_ids, E)
        u = g.fp8_grouped_mm(g.moe_gather(q, o), qg, o.group_rows, act="silu", b_up=qu)
        return q, h, u, o, g.moe_combine(g.fp8_grouped_mm(u, qd, o.group_rows), o, w)

    def check(q, h, u, o, y):
        a = g.fp8_dequantize(q, dtype=torch.float32).double().cpu()
        rows = o.rows.cpu()
        v, size = torch.zeros(T, D, dtype=torch.float64), torch.zeros(T, D, dtype=torch.float64)
        mats = [[torch.from_numpy(held64(m[e].t())).t() for e in range(E)] for m in (gate, up, down)]
        for t in range(T):
            for j in range(top):
                e = int(ids[t, j])
                if 0 <= e < E:
                    z = torch.nn.functional.silu(a[t] @ mats[0][e]) * (a[t] @ mats[1][e])
                    got = u[rows[t, j]].double().cpu()
                    assert ((got - z).abs() <= 2.0 ** -10 * z.abs() + 1e-5).all()
                    part = torch.from_numpy(held64(u[rows[t, j]:rows[t, j] + 1])) @ mats[2][e]
                    v[t] += w[t, j].double().cpu() * part[0]
                    size[t] += (w[t, j].double().cpu() * part[0]).abs()
        # each part is rounded to fp16 once, and their sum
        assert ((y.double().cpu() - v).abs() <= 2.0 ** -11 * (size + v.abs()) + 2.0 ** -14 * size + 1e-4).all()

    ref = layer()
    check(*ref)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        again = layer()
    s.synchronize()
    assert torch.equal(again[4], ref[4])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = layer()
    ids = _ids(T, top, E, 13, 0.5)
    dev_ids.copy_(ids)
    x.mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    check(*kept)
    assert g.gemm_f16_device_status() == 0
