"""The mixture-of-experts layer for a few tokens against its definition in 64 bits.

Tolerances follow the arithmetic: an fp32 sum of exact products is off by at
most 2^-20 of the sum of their magnitudes (any order, a few roundings at the
largest partial sum each), a hidden value by that through the activation (slope
at most 1.13) and the other factor plus its 2^-21 as two fp16 halves, a routing
weight by twice its logit's error plus 2^-20, and y by one rounding to fp16.
With MXFP4 weights the tokens and the hidden values are held as 6 MXFP4 columns:
each leaves at most 1/5 of the largest remainder of its block of 32, so a value
is off by at most 5^-6 of its block's largest magnitude.
"""
import pytest
import torch

import dense_tiled_gemm_fp16_gb300 as g
from tests.mxf4_reference import dequantize64, quantize64

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
ACT64 = {"none": lambda v: v, "relu": torch.relu, "silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu}


def make(T, D, F, E, seed, integers=False):
    gen = torch.Generator().manual_seed(seed)

    def rnd(*shape, scale=1.0):
        if integers:
            return torch.randint(-1, 2, shape, generator=gen).half()
        return (torch.randn(shape, generator=gen) * scale).half()

    return (rnd(T, D), rnd(D, E, scale=D ** -0.5), rnd(E, D, F, scale=D ** -0.5), rnd(E, D, F, scale=D ** -0.5),
            rnd(E, F, D, scale=F ** -0.5))


def stored(w, layout):
    """w on the device in one of the layouts a caller may hold it in."""
    if layout == "kn":
        return w.to(DEV)
    if layout == "nk":
        return w.transpose(1, 2).contiguous().to(DEV).transpose(1, 2)
    if layout == "pitched":   # contracted axis contiguous, rows 8 values apart more than they hold
        e, r, c = w.shape
        buf = torch.full((e, c, -(-r // 8) * 8 + 8), float("nan"), dtype=torch.float16, device=DEV)
        buf[:, :, :r] = w.transpose(1, 2).to(DEV)
        return buf[:, :, :r].transpose(1, 2)
    assert layout == "every"   # no unit stride at all
    buf = torch.full(tuple(w.shape) + (2,), float("nan"), dtype=torch.float16, device=DEV)
    buf[..., 0] = w.to(DEV)
    return buf[..., 0]


def held(w):
    """(the Mxf4Matrix of [E, in, out] along in, its values in 64 bits)."""
    vals = torch.stack([torch.from_numpy(dequantize64(*quantize64(m.double().t().numpy()))[:, :m.shape[0]]).t()
                        for m in w])
    return g.mxf4_quantize(w.to(DEV), axis=-2), vals


def held_error(v, columns):
    """What each value of a narrow side held in MXFP4 columns may be off by."""
    if not columns:
        return torch.zeros_like(v)
    pad = torch.nn.functional.pad(v.abs(), (0, -v.shape[-1] % 32)).view(-1, 32)
    return (5.0 ** -6 * pad.max(dim=1, keepdim=True).values.expand(-1, 32)).reshape(-1)[:v.shape[-1]]


def check(x, router, gate, up, down, top, act, renorm, got, columns=False):
    """x .. down on the CPU (weights as the values they stand for); `columns`: MXFP4 weights."""
    y, w, ids = (t.cpu() for t in got)
    T, E = x.shape[0], router.shape[1]
    x, router, gate, up, down = (t.double() for t in (x, router, gate, up, down))
    l, lmag = x @ router, x.abs() @ router.abs()
    order = torch.argsort(-l, dim=1, stable=True)
    assert y.dtype == torch.float16 and w.dtype == torch.float32 and ids.dtype == torch.int32
    assert tuple(w.shape) == tuple(ids.shape) == (T, top)
    ranked = torch.gather(l, 1, order)
    tol_l = 2.0 ** -20 * lmag.max(dim=1).values
    for t in range(T):
        clear = (ranked[t, :-1] - ranked[t, 1:])[:top] > 2 * tol_l[t]
        if bool(clear.all()):
            assert torch.equal(ids[t].long(), order[t, :top]), t
    chosen = torch.gather(l, 1, ids.long())
    p = torch.softmax(l, dim=1).gather(1, ids.long())
    ref_w = torch.softmax(chosen, dim=1) if renorm else p
    tol_w = ref_w * (2 * tol_l[:, None] + 2.0 ** -20)
    assert ((w.double() - ref_w).abs() <= tol_w).all()
    for t in range(T):
        ref, tol = torch.zeros(x.shape[1], dtype=torch.float64), torch.zeros(x.shape[1], dtype=torch.float64)
        for j in range(top):
            e = int(ids[t, j])
            a, u = x[t] @ gate[e], x[t] @ up[e]
            dx = held_error(x[t], columns)
            da = 2.0 ** -20 * (x[t].abs() @ gate[e].abs()) + dx @ gate[e].abs()
            du = 2.0 ** -20 * (x[t].abs() @ up[e].abs()) + dx @ up[e].abs()
            f = ACT64[act](a)
            h = f * u
            dh = 1.13 * da * (u.abs() + du) + du * f.abs() + 2.0 ** -20 * h.abs() + 2.0 ** -24 + held_error(h, columns)
            o, omag = h @ down[e], h.abs() @ down[e].abs()
            ref += ref_w[t, j] * o
            tol += ref_w[t, j] * (dh @ down[e].abs() + 2.0 ** -20 * omag) + tol_w[t, j] * o.abs()
        tol = tol + 2.0 ** -11 * (ref.abs() + tol) + 2.0 ** -24
        err = (y[t].double() - ref).abs()
        assert (err <= tol).all(), (t, float((err / tol).max()))


SHAPES = [  # T, D, F, E, top
    (1, 64, 64, 1, 1), (1, 8, 8, 2, 2), (1, 7, 5, 3, 2), (1, 2048, 768, 8, 4), (2, 130, 70, 33, 8), (3, 257, 129, 5, 1),
    (7, 512, 320, 64, 8), (8, 1000, 200, 40, 3), (9, 256, 128, 4, 4), (16, 512, 512, 16, 2), (17, 384, 96, 2, 1),
    (33, 200, 136, 100, 8), (64, 512, 256, 8, 8), (64, 320, 192, 512, 8), (40, 96, 64, 1, 1)]


@pytest.mark.parametrize("T,D,F,E,top", SHAPES)
@pytest.mark.parametrize("layout", ["nk", "kn", "mxf4"])
def test_layer(T, D, F, E, top, layout):
    x, router, gate, up, down = make(T, D, F, E, T * 31 + D + E)
    renorm, act = (T + E) % 2 == 0, ("silu", "gelu", "relu")[T % 3]
    if layout == "mxf4":
        dev, vals = zip(*(held(w) for w in (gate, up, down)))
    else:
        dev, vals = [stored(w, layout) for w in (gate, up, down)], (gate, up, down)
    got = g.moe_few(x.to(DEV), router.to(DEV), *dev, top, act=act, renormalize=renorm)
    check(x, router, *vals, top, act, renorm, got, columns=layout == "mxf4")
    again = g.moe_few(x.to(DEV), router.to(DEV), *dev, top, act=act, renormalize=renorm)
    assert all(torch.equal(a, b) for a, b in zip(got, again))   # no order of arrival in the result
    assert g.gemm_f16_device_status() == 0


@pytest.mark.parametrize("layout", ["pitched", "every"])
@pytest.mark.parametrize("T,D,F,E,top", [(1, 72, 40, 4, 2), (12, 250, 130, 6, 3)])
def test_other_layouts(T, D, F, E, top, layout):
    x, router, gate, up, down = make(T, D, F, E, 5)
    xd = torch.zeros((T, 2 * D + 1), dtype=torch.float16, device=DEV)
    xd[:, 1::2] = x.to(DEV)
    rd = router.t().contiguous().to(DEV).t()
    out = torch.full((T, D + 3), -7.0, dtype=torch.float16, device=DEV)
    got = g.moe_few(xd[:, 1::2], rd, *(stored(w, layout) for w in (gate, up, down)), top, out=out[:, 1:D + 1])
    check(x, router, gate, up, down, top, "silu", True, got)
    assert (out[:, 0] == -7).all() and (out[:, D + 1:] == -7).all()


@pytest.mark.parametrize("layout", ["rows", "columns", "every"])
@pytest.mark.parametrize("D,E", [(64, 32), (100, 33), (999, 512), (4096, 7), (520, 96)])
def test_router_layouts(D, E, layout):
    x, router, gate, up, down = make(11, D, 16, E, D + E)
    top = min(8, E)
    if layout == "columns":
        rd = router.t().contiguous().to(DEV).t()
    elif layout == "every":
        rd = torch.zeros((D, E, 3), dtype=torch.float16, device=DEV)
        rd[..., 1] = router.to(DEV)
        rd = rd[..., 1]
    else:
        rd = router.to(DEV)
    got = g.moe_few(x.to(DEV), rd, *(stored(w, "nk") for w in (gate, up, down)), top, renormalize=False)
    check(x, router, gate, up, down, top, "silu", False, got)


@pytest.mark.parametrize("layout", ["nk", "kn", "mxf4"])
@pytest.mark.parametrize("T", [1, 6, 30])
def test_integers_are_exact(T, layout):
    """One expert a token and weights 1: small integers pass every step unrounded."""
    D, F, E = 96, 40, 3
    x, _, gate, up, down = make(T, D, F, E, T, integers=True)
    router = torch.zeros((D, E)).half()
    router[0] = torch.tensor([0.0, 1.0, 2.0])
    x[:, 0] = torch.tensor([1.0, -1.0])[torch.arange(T) % 2].half()
    dev = [held(w)[0] if layout == "mxf4" else stored(w, layout) for w in (gate, up, down)]
    y, w, ids = g.moe_few(x.to(DEV), router.to(DEV), *dev, 1, act="relu")
    pick = torch.where(x[:, 0] > 0, 2, 0)
    assert torch.equal(ids[:, 0].cpu().long(), pick) and (w == 1).all()
    ref = torch.stack([(torch.relu(x[t].double() @ gate[e].double()) * (x[t].double() @ up[e].double())) @ down[e].double()
                       for t, e in enumerate(pick.tolist())])
    assert ref.abs().max() <= 2048 * 4 and torch.equal(y.cpu().double(), ref.half().double())


def test_equal_logits_go_to_the_lower_index():
    x, router, gate, up, down = make(10, 128, 32, 70, 3)
    router = router[:, torch.arange(70) % 7].contiguous()   # experts e and e + 7 have equal logits
    _, _, ids = g.moe_few(x.to(DEV), router.to(DEV), *(stored(w, "nk") for w in (gate, up, down)), 8)
    first = (x.double() @ router[:, :7].double()).argmax(dim=1)
    assert torch.equal(ids.cpu().long(), first[:, None] + 7 * torch.arange(8))
    zero = torch.zeros_like(router)
    _, w, ids = g.moe_few(x.to(DEV), zero.to(DEV), *(stored(w, "nk") for w in (gate, up, down)), 5, renormalize=False)
    assert torch.equal(ids.cpu().long(), torch.arange(5).expand(10, 5)) and torch.allclose(w.cpu(), torch.tensor(1 / 70))


@pytest.mark.parametrize("layout", ["nk", "mxf4"])
def test_infinities_and_nan_stay_with_their_token(layout):
    x, router, gate, up, down = make(6, 256, 100, 9, 8)
    dev = [held(w)[0] if layout == "mxf4" else stored(w, layout) for w in (gate, up, down)]
    ref = g.moe_few(x.to(DEV), router.to(DEV), *dev, 3)
    bad = x.clone()
    bad[1, 7], bad[4, 200] = float("nan"), float("inf")
    got = g.moe_few(bad.to(DEV), router.to(DEV), *dev, 3)
    keep = torch.tensor([0, 2, 3, 5], device=DEV)
    for a, b in zip(got, ref):
        assert torch.equal(a[keep], b[keep])
    assert torch.isnan(got[0][1]).all() and not torch.isfinite(got[0][4]).any()
    assert torch.isnan(got[1][1]).all()


def test_an_unread_expert_may_hold_anything():
    x, router, gate, up, down = make(4, 128, 64, 6, 2)
    router[:, 5] = 0
    x[:, 0], router[0, :5], router[0, 5] = 4.0, 4.0, -4.0
    dev = [stored(w, "nk") for w in (gate, up, down)]
    ref = g.moe_few(x.to(DEV), router.to(DEV), *dev, 5)
    for w in dev:
        w[5] = float("nan")
    got = g.moe_few(x.to(DEV), router.to(DEV), *dev, 5)
    assert (ref[2] != 5).all() and all(torch.equal(a, b) for a, b in zip(got, ref))


def test_hidden_values_past_fp16_become_infinite():
    x = torch.full((1, 8), 100.0).half()
    one = torch.ones((1, 8, 8)).half()
    y, _, _ = g.moe_few(x.to(DEV), torch.ones((8, 1)).half().to(DEV), *(one.to(DEV) for _ in range(3)), 1, act="none")
    assert torch.isinf(y).all() and (y > 0).all()


def test_streams_and_a_graph():
    x, router, gate, up, down = (t.to(DEV) for t in make(5, 512, 256, 16, 1))
    ref = g.moe_few(x, router, gate, up, down, 4)
    other = g.moe_few(-x, router, gate, up, down, 4)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs, neg = [], -x
    torch.cuda.synchronize()
    for _ in range(20):
        for i, s in enumerate(streams):
            outs.append((i, g.moe_few(neg if i % 2 else x, router, gate, up, down, 4, stream=s)))
    torch.cuda.synchronize()
    for i, got in outs:
        assert all(torch.equal(a, b) for a, b in zip(got, other if i % 2 else ref))
    graph = torch.cuda.CUDAGraph()
    buf = x.clone()
    with torch.cuda.graph(graph):
        got = g.moe_few(buf, router, gate, up, down, 4)
    for want, value in ((other, neg), (ref, x)):
        buf.copy_(value)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert g.gemm_f16_device_status() == 0


def test_stalled_wait_reports_timeout_and_the_context_survives():
    x, router, gate, up, down = (t.to(DEV) for t in make(3, 256, 128, 8, 4))
    ref = g.moe_few(x, router, gate, up, down, 2)
    g.gemm_f16_device_status(reset=True)
    try:
        g.gemm_f16_set_option(g.OPT_TIMEOUT_MS, 50)
        g.gemm_f16_set_option(g.OPT_TEST_STALL, 1)
        g.moe_few(x, router, gate, up, down, 2)
        assert g.gemm_f16_device_status(reset=True) == g.ERR_TIMEOUT
    finally:
        g.gemm_f16_set_option(g.OPT_TEST_STALL, 0)
        g.gemm_f16_set_option(g.OPT_TIMEOUT_MS, 0)
    assert all(torch.equal(a, b) for a, b in zip(g.moe_few(x, router, gate, up, down, 2), ref))
    assert g.gemm_f16_device_status() == 0
