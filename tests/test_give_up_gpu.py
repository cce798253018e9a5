"""A wait that runs out ends the MXFP4 product and the expert layer with a status, in every form of
theirs, and leaves the context usable.  The kernels' own stall option makes a bounded wait run out."""
import contextlib

import pytest
import torch

import dense_tiled_gemm_fp16_gb300 as g
from tests.test_moe_gpu import make, stored
from tests.test_moe_hidden_gpu import stored as stored_at

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


# few rows without and with a cluster, few columns, split along K, pairs of either width
@pytest.mark.parametrize("M,N,K", [(3, 260, 1024), (16, 520, 8192), (1000, 16, 4096), (100, 200, 16384), (300, 300, 512),
                                   (3001, 2000, 300)])
@pytest.mark.parametrize("a16", [False, True])
def test_product(M, N, K, a16):
    gen = torch.Generator().manual_seed(M)
    x, w = (torch.randn((r, K), generator=gen).half().to(DEV) for r in (M, N))
    q = g.mxf4_quantize(w)
    a = x if a16 else g.mxf4_quantize(x)
    ref = g.mxf4_mm(a, q)
    with stalled():
        g.mxf4_mm(a, q)
    assert torch.equal(g.mxf4_mm(a, q), ref) and g.gemm_f16_device_status() == 0


@pytest.mark.parametrize("layout", ["nk", "kn", "mxf4", "odd rows", "odd columns", "every"])
@pytest.mark.parametrize("T", [3, 12, 50])
def test_experts(T, layout):
    x, router, gate, up, down = make(T, 264, 136, 8, 4)
    if layout == "mxf4":
        ws = [g.mxf4_quantize(w.to(DEV), axis=-2) for w in (gate, up, down)]
    else:
        ws = [(stored if layout in ("nk", "kn", "every") else stored_at)(w, layout) for w in (gate, up, down)]
    args = (x.to(DEV), router.to(DEV), *ws, 3)
    ref = g.moe_few(*args)
    with stalled():
        g.moe_few(*args)
    assert all(torch.equal(a, b) for a, b in zip(g.moe_few(*args), ref)) and g.gemm_f16_device_status() == 0
