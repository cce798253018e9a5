"""The 8-bit products, the norm and the expert order at their ends: waits that run out, offsets past 32 bits,
other streams and places, graphs that share nothing, repeated calls.

A stalled wait is made by the kernels' own option: a barrier that nothing arrives on, given up after 50 ms.
"""
import contextlib

import pytest
import torch

import dense_tiled_gemm_fp16_gb300 as g

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


@contextlib.contextmanager
def stalled():
    g.gemm_f16_device_status(reset=True)
    try:
        g.gemm_f16_set_option(g.OPT_TIMEOUT_MS, 50)
        g.gemm_f16_set_option(g.OPT_TEST_STALL, 1)
        yield
        assert g.gemm_f16_device_status(reset=True) == g.ERR_TIMEOUT
    finally:
        g.gemm_f16_set_option(g.OPT_TEST_STALL, 0)
        g.gemm_f16_set_option(g.OPT_TIMEOUT_MS, 0)
        g.gemm_f16_set_option(g.OPT_PAIR, 0)


def _x(*shape, seed=0, dtype=torch.float16):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    return torch.empty(shape, dtype=dtype, device=DEV).normal_(generator=gen)


@pytest.mark.parametrize("M,N,K,form", [(16, 512, 4096, 1), (300, 200, 700, 1), (300, 700, 2000, 2), (2000, 3000, 512, 2)])
def test_a_wait_that_runs_out_ends_a_product(M, N, K, form):
    a, b = _x(M, K), g.fp8_quantize(_x(N, K, seed=1))
    g.gemm_f16_set_option(g.OPT_PAIR, form)
    ref = g.fp8_mm(a, b)
    with stalled():
        g.gemm_f16_set_option(g.OPT_PAIR, form)
        g.fp8_mm(a, b)
    g.gemm_f16_set_option(g.OPT_PAIR, form)
    assert torch.equal(g.fp8_mm(a, b), ref)
    g.gemm_f16_set_option(g.OPT_PAIR, 0)
    assert g.gemm_f16_device_status() == 0


@pytest.mark.parametrize("gated", [False, True])
def test_a_wait_that_runs_out_ends_a_grouped_product(gated):
    a, b, u = _x(700, 600), g.fp8_quantize(_x(5, 300, 600, seed=1)), g.fp8_quantize(_x(5, 300, 600, seed=2))
    counts = torch.tensor([300, 0, 150, 200, 50], dtype=torch.int32, device=DEV)
    call = lambda: g.fp8_grouped_mm(a, b, counts, act="silu", b_up=u if gated else None)  # noqa: E731
    ref = call()
    with stalled():
        call()
    assert torch.equal(call(), ref)
    assert g.gemm_f16_device_status() == 0


@pytest.fixture
def pairs():
    """The pair kernel alone, which sums each output's K in order (the small form cuts K by the number of
    tiles, so that its sums of other shapes round differently)."""
    g.gemm_f16_set_option(g.OPT_PAIR, 2)
    yield
    g.gemm_f16_set_option(g.OPT_PAIR, 0)


def test_offsets_past_32_bits(pairs):
    """4.9e9 values: the last rows equal those of a call on them alone."""
    R, d, tail = 600_000, 8192, 300
    x = torch.empty((R, d), dtype=torch.float16, device=DEV).normal_(generator=torch.Generator(device=DEV).manual_seed(0))
    w, b = _x(d, seed=1), g.fp8_quantize(_x(48, d, seed=2))
    q = g.rms_norm(x, w, quantize=True)
    last = x[-tail:].clone()
    ref = g.rms_norm(last, w, quantize=True)
    assert torch.equal(g.fp8_mm(q, b)[-tail:], g.fp8_mm(ref, b))
    back = g.fp8_dequantize(q)
    assert torch.equal(back[-tail:], g.fp8_dequantize(ref))
    del back
    y = g.rms_norm(x, w)
    assert torch.equal(y[-tail:], g.rms_norm(last, w))
    q2 = g.fp8_quantize(y)
    assert torch.equal(g.fp8_mm(q2, b)[-tail:], g.fp8_mm(g.fp8_quantize(y[-tail:]), b))
    del q, q2
    # as a grouped product whose last group begins past 2^32 bytes of A
    counts = torch.tensor([R - 123, 123], dtype=torch.int32, device=DEV)
    two = g.fp8_quantize(torch.stack([_x(48, d, seed=2), _x(48, d, seed=3)]))
    out = g.fp8_grouped_mm(y, two, counts)
    one = g.fp8_quantize(_x(48, d, seed=3))
    assert torch.equal(out[-123:], g.fp8_mm(y[-123:], one)) and torch.equal(out[:100], g.fp8_mm(y[:100], b))


def test_rows_past_32_bits_in_the_experts_order():
    T, top, d = 150_000, 4, 8192
    ids = torch.arange(T * top, device=DEV, dtype=torch.int32).view(T, top) % 4
    o = g.moe_sort(ids, 4)
    x = torch.empty((T, d), dtype=torch.float16, device=DEV).normal_(generator=torch.Generator(device=DEV).manual_seed(0))
    xs = g.moe_gather(x, o)
    assert xs.numel() > 2 ** 32 and torch.equal(xs[-1000:], x[-1000:]) and torch.equal(xs[:1000], x[:1000])
    w = torch.full((T, top), 0.25, device=DEV)
    assert torch.equal(g.moe_combine(xs, o, w), x)
    dy, dw = g.moe_combine_grad(x, xs, o, w)
    assert torch.equal(dy[-1000:], 0.25 * x[-1000:])
    assert torch.allclose(dw[-5:, 2].double(), x[-5:].double().square().sum(dim=1), rtol=1e-5)


def test_graphs_that_share_nothing():
    """Two captured steps, replayed at once on two streams: each keeps its own workspace."""
    T, E, top, D, F = 200, 6, 2, 512, 384
    gate, up, down = (g.fp8_quantize(_x(E, *s, seed=i)) for i, s in enumerate(((F, D), (F, D), (D, F))))
    w = torch.ones(D, dtype=torch.float16, device=DEV)

    def step(x, ids, weights):
        o = g.moe_sort(ids, E)
        h = g.fp8_grouped_mm(g.moe_gather(g.rms_norm(x, w, quantize=True), o), gate, o.group_rows, act="silu", b_up=up)
        return g.moe_combine(g.fp8_grouped_mm(h, down, o.group_rows), o, weights)

    inputs, refs, graphs, outs = [], [], [], []
    for k in range(2):
        gen = torch.Generator(device=DEV).manual_seed(k)
        args = (_x(T * (9 * k + 1), D, seed=10 + k), torch.randint(0, E, (T * (9 * k + 1), top), generator=gen, device=DEV).int(),
                torch.rand((T * (9 * k + 1), top), generator=gen, device=DEV))
        refs.append(step(*args))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(step(*args))
        inputs.append(args), graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(10):
        for s, graph in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, refs))


def test_plain_stream_order():
    """Without programmatic launches the results are the same."""
    a, b = _x(40, 900), g.fp8_quantize(_x(700, 900, seed=1))
    ref = g.fp8_mm(a, b)
    try:
        g.gemm_f16_set_option(g.OPT_PDL, 1)
        assert torch.equal(g.fp8_mm(a, b), ref)
    finally:
        g.gemm_f16_set_option(g.OPT_PDL, 0)


@pytest.mark.parametrize("width", [64, 128, 192, 256])
def test_forced_widths(width):
    a, b = _x(1000, 700), g.fp8_quantize(_x(3, 520, 700, seed=1))
    counts = torch.tensor([600, 1, 399], dtype=torch.int32, device=DEV)
    ref = g.fp8_grouped_mm(a, b, counts)
    try:
        g.gemm_f16_set_option(g.OPT_TILE_N, width)
        assert torch.equal(g.fp8_grouped_mm(a, b, counts), ref)   # a sum's order does not hang on its tile
    finally:
        g.gemm_f16_set_option(g.OPT_TILE_N, 0)


def test_the_same_call_gives_the_same_bits():
    x, w = _x(3000, 7168), _x(7168, seed=1)
    b = g.fp8_quantize(_x(2048, 7168, seed=2))
    ids = torch.randint(0, 64, (3000, 8), device=DEV).int()
    first = None
    for _ in range(5):
        o = g.moe_sort(ids, 64)
        q = g.rms_norm(x, w, quantize=True)
        c = g.fp8_mm(q, b)
        y = g.moe_combine(g.moe_gather(c, o), o, torch.ones((3000, 8), device=DEV) / 8)
        now = [o.order, q.codes.clone(), c, y]
        assert first is None or all(torch.equal(a, b) for a, b in zip(first, now))
        first = now
