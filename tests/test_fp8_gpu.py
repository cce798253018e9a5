"""8-bit matrices and their products against 64 bits.

Quantisation and its inverse are exact: codes and scales equal the definition's, values are rounded
once.  Products: an instruction takes 32 values of k and rounds the sum once, so a sum is off by at
most ceil(K / 32) + 1 times 2^-23 of the sum of its terms' magnitudes; an activation adds its slope (at most
1.13) of that and 2^-18 of its own value, a product of two such sums both, and the result is rounded
once (2^-11 of it in fp16, 2^-25 where it is subnormal; 2^-8 in bf16).
"""
import numpy as np
import pytest
import torch

import dense_tiled_gemm_fp16_gb300 as g
from tests.fp8_reference import codes_plain, dequantize64, held64, quantize64, scales_plain

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
TYPES = [torch.float16, torch.bfloat16, torch.float32]


@pytest.fixture(autouse=True)
def _clean():
    yield
    g.gemm_f16_set_option(g.OPT_PAIR, 0)
    assert g.gemm_f16_device_status() == 0


def _arrays(q):
    torch.cuda.synchronize()
    b = q.batch or 1
    c, s = q.codes.cpu().numpy().reshape(b, -1), q.scales.cpu().numpy().reshape(b, -1)
    return [(codes_plain(c[i], q.rows, q.k), scales_plain(s[i], q.rows, q.k)) for i in range(b)]


def _same(q, x):
    """q holds the matrices x (of [.., rows, k]) exactly as the definition says."""
    mats = x.double().cpu().numpy().reshape(q.batch or 1, q.rows, q.k)
    for (c, s), m in zip(_arrays(q), mats):
        rc, rs = quantize64(m)
        assert (s == rs).all()
        assert (c == rc[:, :q.k]).all()


def _values(shape, seed, dtype):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=gen) * torch.exp2(torch.randint(-9, 9, shape[:-1] + (1,), generator=gen).float())
    x[torch.rand(shape, generator=gen) < 0.1] *= 2.0 ** -8
    return x.to(dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,k", [(1, 1), (1, 128), (3, 129), (16, 8192), (128, 512), (129, 513), (300, 70), (1000, 1023),
                                    (5000, 4097)])
def test_quantize_and_back(rows, k, dtype):
    x = _values((rows, k), rows + k, dtype)
    q = g.fp8_quantize(x.to(DEV))
    _same(q, x)
    v = dequantize64(*quantize64(x.double().numpy()))[:, :k]
    for to in TYPES:
        assert torch.equal(g.fp8_dequantize(q, dtype=to).cpu(), torch.from_numpy(v).to(to))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("batch,rows,k", [(1, 9, 513), (9, 9, 5000), (1, 1281, 4100), (31, 33, 5000), (1, 5153, 4104)])
def test_quantize_rows_a_block(batch, rows, k, dtype):
    """Blocks of 8, 16 and 32 rows, the last of them with one row."""
    x = _values((batch, rows, k), batch + rows + k, dtype)
    _same(g.fp8_quantize(x.to(DEV)), x)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,k", [(1, 300), (77, 1), (129, 513), (1000, 640)])
def test_quantize_strided(rows, k, dtype):
    x = _values((rows, k), rows + k, dtype).to(DEV)
    _same(g.fp8_quantize(x.t().contiguous().t()), x)                   # transposed
    _same(g.fp8_quantize(x.t().contiguous(), axis=-2), x)              # a weight [k, rows]
    wide = torch.zeros((2 * rows, 3 * k + 1), dtype=dtype, device=DEV)
    wide[::2, 1::3] = x
    _same(g.fp8_quantize(wide[::2, 1::3]), x)                          # neither stride one
    off = torch.zeros((rows, k + 3), dtype=dtype, device=DEV)
    off[:, 3:] = x
    _same(g.fp8_quantize(off[:, 3:]), x)                               # rows that start anywhere


def test_quantize_batches():
    x = _values((3, 130, 520), 5, torch.float16).to(DEV)
    _same(g.fp8_quantize(x), x)
    _same(g.fp8_quantize(x.transpose(1, 2), axis=1), x)
    _same(g.fp8_quantize(x[:1].expand(4, -1, -1)), x[:1].expand(4, -1, -1))
    _same(g.fp8_quantize(torch.empty((1, 130, 520), dtype=torch.float16, device=DEV).copy_(x[:1])), x[:1])


def test_every_rounding_point_and_special_values():
    """All e4m3 numbers, the points between neighbours and their fp32 neighbours; the scale's own border; NaN
    and infinity take their block alone; magnitudes at the types' ends."""
    from tests.fp8_reference import GRID
    mid = (GRID[1:] + GRID[:-1]) / 2
    pts = np.concatenate([GRID, mid]).astype(np.float32)
    pts = np.concatenate([pts, np.nextafter(pts, np.float32(np.inf)), np.nextafter(pts, np.float32(0))])
    pts = pts[pts <= 448]
    x = torch.zeros((2, 128 * len(pts)))
    for sign in (0, 1):
        rows = x[sign].view(-1, 128)
        rows[:, 0] = 448.0   # the scale is 2^0
        rows[:, 1:] = torch.from_numpy(pts).unsqueeze(1) * (1 - 2 * sign)
    _same(g.fp8_quantize(x.to(DEV)), x)
    _same(g.fp8_quantize((x[:, ::7] * 2.0 ** 100).contiguous().to(DEV)), x[:, ::7] * 2.0 ** 100)
    for dtype in TYPES:
        big, tiny = torch.finfo(dtype).max, torch.finfo(dtype).smallest_normal
        v = torch.zeros((9, 256), dtype=dtype)
        for i, top in enumerate((448, 449, 1.75, 1.7578125, big, tiny, tiny / 4, 0, 1)):
            v[i, 3], v[i, 200] = top, -top
        v[8, 5], v[7, 130] = float("inf"), float("nan")
        q = g.fp8_quantize(v.to(DEV))
        _same(q, v)
        back = g.fp8_dequantize(q, dtype=torch.float32).cpu()
        assert back[8, :128].isnan().all() and not back[8, 128:].isnan().any()
        assert back[7, 128:].isnan().all() and not back[7, :128].isnan().any()


def _operands(M, N, K, seed, dtype, scale=1.0):
    gen = torch.Generator().manual_seed(seed)
    x = (torch.randn((M, K), generator=gen) * scale).to(dtype)
    w = (torch.randn((N, K), generator=gen) * K ** -0.5).to(dtype)
    return x, w


def _act(name, v):
    f = torch.nn.functional
    v = torch.from_numpy(v)
    return {"none": lambda t: t, "relu": torch.relu, "silu": f.silu, "gelu": f.gelu}[name](v).numpy()


def _near(c, sums, sizes, K, act="none"):
    """c holds act(sums[0]) (times sums[1]) to the tolerance above; sizes: sums of the terms' magnitudes."""
    step = (-(-K // 32) + 1) * 2.0 ** -23
    v, tol = sums[0], step * sizes[0]
    if act != "none":
        v = _act(act, v)
        tol = 1.13 * tol + 2.0 ** -18 * np.abs(v)
    if len(sums) > 1:
        tol = tol * (np.abs(sums[1]) + step * sizes[1]) + np.abs(v) * step * sizes[1]
        v = v * sums[1]
    half = c.dtype is torch.float16
    tol = tol + (2.0 ** -11 * np.abs(v) + 2.0 ** -25 if half else 2.0 ** -8 * np.abs(v))
    err = np.abs(c.cpu().double().numpy() - v)
    assert (err <= tol).all(), (np.argwhere(err > tol)[:5], (err / tol).max())


SHAPES = [(1, 16, 1), (1, 300, 128), (3, 129, 130), (16, 1000, 4097), (33, 512, 1024), (64, 64, 70), (65, 257, 513),
          (100, 31, 700), (300, 4096, 600), (700, 2003, 300), (1500, 1999, 130), (2000, 64, 1000), (129, 6000, 2100)]


@pytest.mark.parametrize("dtype", TYPES[:2])
@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("form", [0, 1, 2])
def test_products(M, N, K, dtype, form):
    """Either kernel on every shape, and the library's own choice; A held and A quantised within the call."""
    x, w = _operands(M, N, K, M + N + K, dtype)
    a, b = held64(x), held64(w)
    g.gemm_f16_set_option(g.OPT_PAIR, form)
    qw = g.fp8_quantize(w.to(DEV))
    c = g.fp8_mm(x.to(DEV), qw, dtype=dtype)
    _near(c, [a @ b.T], [np.abs(a) @ np.abs(b).T], K)
    assert torch.equal(c, g.fp8_mm(g.fp8_quantize(x.to(DEV)), qw, dtype=dtype))


@pytest.mark.parametrize("form", [1, 2])
@pytest.mark.parametrize("M,N,K", [(17, 300, 200), (301, 511, 300), (300, 512, 640)])
@pytest.mark.parametrize("act,scale", [("none", 1), ("relu", 1), ("silu", 8), ("gelu", 2.5)])
@pytest.mark.parametrize("lead,pitch", [(0, 8), (3, 5)])
def test_bias_activation_and_the_output_s_place(M, N, K, act, scale, lead, pitch, form):
    for dtype in TYPES[:2]:
        x, w = _operands(M, N, K, M + N + K, dtype, scale)
        bias = torch.randn(N, generator=torch.Generator().manual_seed(3)).to(dtype)
        ld = (N + 7) // 8 * 8 + pitch
        buf = torch.full((M + 2, ld), -7.0, dtype=dtype, device=DEV)
        out = buf[1:M + 1, lead:lead + N]
        g.gemm_f16_set_option(g.OPT_PAIR, form)
        g.fp8_mm(x.to(DEV), g.fp8_quantize(w.to(DEV)), bias=bias.to(DEV), act=act, out=out)
        a, b, v = held64(x), held64(w), bias.double().numpy()
        _near(out, [a @ b.T + v], [np.abs(a) @ np.abs(b).T + np.abs(v)], K, act)
        out.fill_(-7.0)
        assert (buf == -7.0).all()   # nothing around the output was written


def test_a_block_with_a_nan_reaches_its_row_and_nothing_else():
    x, w = _operands(70, 300, 400, 1, torch.float16)
    x[5, 130], x[40, 399] = float("nan"), float("-inf")
    for form in (1, 2):
        g.gemm_f16_set_option(g.OPT_PAIR, form)
        c = g.fp8_mm(x.to(DEV), g.fp8_quantize(w.to(DEV)))
        rows = c.isnan().any(dim=1).nonzero().flatten().tolist()
        assert rows == [5, 40] and c[rows].isnan().all()


def _groups(kind, groups, rows, gen):
    if kind == "even":
        return [rows // groups] * groups
    p = torch.rand(groups, generator=gen) ** 3
    p[torch.rand(groups, generator=gen) < 0.3] = 0
    p[groups // 2] += 0.1
    return torch.bincount(torch.multinomial(p, rows, replacement=True, generator=gen), minlength=groups).tolist()


@pytest.mark.parametrize("dtype", TYPES[:2])
@pytest.mark.parametrize("kind", ["even", "uneven"])
@pytest.mark.parametrize("groups,rows,N,K", [(1, 1, 64, 128), (1, 300, 257, 70), (4, 8, 300, 600), (7, 1000, 129, 520),
                                             (64, 512, 256, 640), (5, 2000, 520, 300), (130, 900, 100, 200)])
@pytest.mark.parametrize("gated", [False, True])
def test_grouped(groups, rows, N, K, kind, gated, dtype):
    gen = torch.Generator().manual_seed(groups + rows + N)
    counts = _groups(kind, groups, rows, gen)
    spare = rows - sum(counts) + 3   # rows of no group
    x = torch.randn((sum(counts) + spare, K), generator=gen).to(dtype)
    ws = [(torch.randn((groups, K, N), generator=gen) * K ** -0.5).to(dtype) for _ in range(2 if gated else 1)]
    q = [g.fp8_quantize(w.to(DEV), axis=-2) for w in ws]
    gr = torch.tensor(counts, dtype=torch.int32, device=DEV)
    out = torch.full((x.shape[0], N), -7.0, dtype=dtype, device=DEV)
    act = "silu" if gated else "none"
    g.fp8_grouped_mm(x.to(DEV), q[0], gr, act=act, b_up=q[1] if gated else None, out=out)
    assert (out[sum(counts):] == -7.0).all()
    at = 0
    for i, n in enumerate(counts):
        if n:
            a, bs = held64(x[at:at + n]), [held64(w[i].t()) for w in ws]
            _near(out[at:at + n], [a @ b.T for b in bs], [np.abs(a) @ np.abs(b).T for b in bs], K, act)
        at += n
    again = torch.full_like(out, -7.0)
    g.fp8_grouped_mm(g.fp8_quantize(x.to(DEV)), q[0], gr, act=act, b_up=q[1] if gated else None, out=again)
    assert torch.equal(out, again)


def test_counts_that_the_rows_do_not_hold():
    """Counts below zero are none, rows past the matrix are absent; nothing else is written."""
    K, N = 256, 96
    gen = torch.Generator().manual_seed(8)
    x = torch.randn((50, K), generator=gen).half().to(DEV)
    w = g.fp8_quantize(torch.randn((4, K, N), generator=gen).half().to(DEV), axis=-2)
    buf = torch.full((60, N), -7.0, dtype=torch.float16, device=DEV)
    count = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    ref = g.fp8_grouped_mm(x, w, count(20, 0, 30, 0))
    for v in ((20, -5, 30, 0), (20, -2**31, 2**31 - 1, 2**31 - 1), (20, 0, 1000, 7)):
        g.fp8_grouped_mm(x, w, count(*v), out=buf[:50])
        assert torch.equal(buf[:50], ref) and (buf[50:] == -7.0).all()
    buf.fill_(-7.0)
    g.fp8_grouped_mm(x, w, count(0, 0, 0, 0), out=buf[:50])
    assert (buf == -7.0).all()
    assert g.fp8_grouped_mm(x[:0], w, count(0, 0, 0, 0)).shape == (0, N)


def test_on_a_side_stream_and_in_a_graph():
    x, w = _operands(200, 384, 700, 2, torch.float16)
    x, qw = x.to(DEV), g.fp8_quantize(w.to(DEV))
    qg = g.fp8_quantize(torch.stack([w, -w]).to(DEV))
    counts = torch.tensor([90, 110], dtype=torch.int32, device=DEV)
    ref, refg = g.fp8_mm(x, qw), g.fp8_grouped_mm(x, qg, counts)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c, cg = g.fp8_mm(x, qw, stream=s), g.fp8_grouped_mm(x, qg, counts, stream=s)
    s.synchronize()
    assert torch.equal(c, ref) and torch.equal(cg, refg)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c, cg = g.fp8_mm(x, qw), g.fp8_grouped_mm(x, qg, counts)
    x.mul_(2)
    counts.copy_(torch.tensor([110, 90]))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(c, g.fp8_mm(x, qw)) and torch.equal(cg, g.fp8_grouped_mm(x, qg, counts))
    assert not torch.equal(cg, refg)


def test_two_calls_at_once():
    """Calls on two streams share no memory of the library's."""
    x, w = _operands(600, 700, 1000, 4, torch.float16)
    x, qw = x.to(DEV), g.fp8_quantize(w.to(DEV))
    ref = g.fp8_mm(x, qw)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [g.fp8_mm(x, qw, stream=streams[i % 2]) for i in range(20)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref) for o in outs)
