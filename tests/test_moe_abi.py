"""The mixture-of-experts entry points without a GPU: exports, sizes and refusals."""
import ctypes
import os
import re

import pytest
import torch

import dense_tiled_gemm_fp16_gb300 as g
from dense_tiled_gemm_fp16_gb300 import moe

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# Fake, non-null, aligned "pointers": the calls are refused before any use.
X, R, G, U, DN, Y, W, I, WS = (1 << s for s in range(20, 47, 3))


def _w(data=G, fmt=0, scales=None, se=4096, si=1, so=64):
    return g.MoeWeight(fmt, data, scales, se, si, so)


def _args(**k):
    a = dict(x=X, sxt=64, sxi=1, router=R, sri=4, sre=1, gate=_w(G), up=_w(U), down=_w(DN), T=2, D=64, F=64, E=4, top=2,
             renorm=1, act=2, y=Y, ldy=64, weights=W, ids=I, ws=WS, wb=1 << 24)
    assert set(k) <= set(a)
    return tuple({**a, **k}.values())


def _refused(call, status=g.ERR_INVALID_VALUE):
    with pytest.raises(g.GemmF16Error) as e:
        call()
    assert e.value.status == status


def _header():
    src = open(os.path.join(ROOT, "include", "moe_f16.h")).read()
    return re.sub(r"/\*.*?\*/", "", src, flags=re.S)


def test_every_declared_symbol_is_exported():
    names = set(re.findall(r"\b(moe_f16\w*)\s*\(", _header()))
    assert names == set(moe.EXPORTED)
    for n in names:
        assert ctypes.cast(getattr(g.lib(), n), ctypes.c_void_p).value
    for name, value in re.findall(r"#define MOE_F16_(MAX_\w+) (\d+)", _header()):
        assert getattr(moe, name) == int(value)
    for name, value in re.findall(r"MOE_F16_(WEIGHT_\w+) = (\d)", _header()):
        assert getattr(moe, name) == int(value)


@pytest.mark.parametrize("sizes", [(0, 64, 64, 4, 2), (65, 64, 64, 4, 2), (1, 0, 64, 4, 2), (1, 32769, 64, 4, 2),
                                   (1, 64, 0, 4, 2), (1, 64, 32769, 4, 2), (1, 64, 64, 0, 1), (1, 64, 64, 513, 2),
                                   (1, 64, 64, 4, 0), (1, 64, 64, 4, 5), (1, 64, 64, 16, 9)])
def test_sizes_out_of_range(sizes):
    _refused(lambda: g.moe_f16_workspace_size(*sizes))
    T, D, F, E, top = sizes
    _refused(lambda: g.moe_f16(*_args(T=T, D=D, F=F, E=E, top=top, ldy=1 << 20)))


def test_workspace_grows_with_the_tokens():
    one, many = (g.moe_f16_workspace_size(t, 100, 70, 8, 3) for t in (1, 64))
    assert 0 < one < many and one % 256 == many % 256 == 0
    _refused(lambda: g.moe_f16(*_args(wb=g.moe_f16_workspace_size(2, 64, 64, 4, 2) - 1)), g.ERR_OUT_OF_MEMORY)


@pytest.mark.parametrize("bad", [
    dict(x=0), dict(router=0), dict(y=0), dict(weights=0), dict(ids=0), dict(ws=0), dict(x=X + 1), dict(router=R + 1),
    dict(y=Y + 1), dict(weights=W + 2), dict(ids=I + 2), dict(ws=WS + 16), dict(sxt=0), dict(sxi=-1), dict(sri=0),
    dict(sre=0), dict(ldy=63), dict(act=4), dict(act=-1), dict(gate=_w(0)), dict(up=_w(U + 1)), dict(down=_w(DN, fmt=2)),
    dict(gate=_w(G, se=-1)), dict(gate=_w(G, si=0)), dict(gate=_w(G, so=-8)), dict(gate=_w(G, so=1 << 62)),
    dict(gate=_w(G, scales=WS)),                                    # fp16 weights have no scales
    dict(gate=_w(G, fmt=1, scales=WS)),                             # formats differ
    dict(gate=_w(G, fmt=1), up=_w(U, fmt=1, scales=WS), down=_w(DN, fmt=1, scales=WS)),   # no scales
    dict(gate=_w(G + 8, fmt=1, scales=G + (1 << 16)), up=_w(U, fmt=1, scales=U + (1 << 16)),
         down=_w(DN, fmt=1, scales=DN + (1 << 16)))])
def test_refusals(bad):
    _refused(lambda: g.moe_f16(*_args(**bad)))


@pytest.mark.parametrize("bad", [dict(y=X), dict(y=R), dict(y=G + 64), dict(weights=U), dict(ids=DN + 4), dict(ws=X),
                                 dict(weights=Y), dict(ids=W), dict(ids=WS), dict(y=WS + 256)])
def test_overlaps_are_refused(bad):
    _refused(lambda: g.moe_f16(*_args(**bad)), g.ERR_ALIAS)


def test_a_valid_call_reaches_the_device_check():
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    _refused(lambda: g.moe_f16(*_args()), g.ERR_UNSUPPORTED_DEVICE)


def test_tensor_form_checks_before_any_call():
    h = torch.float16
    z = lambda *s, dtype=h: torch.zeros(s, dtype=dtype)   # noqa: E731
    x, r, gate, down = z(3, 16), z(16, 4), z(4, 16, 8), z(4, 8, 16)
    for bad in ((z(16), r, gate, gate, down), (x, z(15, 4), gate, gate, down), (x, r, z(4, 8, 16), gate, down),
                (x, r, gate, z(4, 16, 9), down), (x, r, gate, gate, z(4, 16, 8)), (x, r, z(3, 16, 8), gate, down),
                (x, r, z(16, 8), gate, down)):
        with pytest.raises(ValueError):
            g.moe_few(*bad, 2)
    with pytest.raises(TypeError):
        g.moe_few(x.float(), r, gate, gate, down, 2)
    with pytest.raises(TypeError):
        g.moe_few(x, r, gate.float(), gate, down, 2)
    q = g.Mxf4Matrix(torch.zeros(4 * 8 * 16, dtype=torch.uint8), torch.zeros(2048, dtype=torch.uint8), 8, 16, 4)
    with pytest.raises(TypeError):                        # one format for the three
        g.moe_few(x, r, q, gate, down, 2)
    with pytest.raises(ValueError):                       # quantised along the wrong axis
        g.moe_few(x, r, q, q, q, 2)
    with pytest.raises(ValueError):
        g.moe_few(x, r, gate, gate, down, 2, act="tanh")
    with pytest.raises(ValueError):
        g.moe_few(x, r, gate, gate, down, 2, out=z(3, 15))
    with pytest.raises(ValueError):                       # host tensors
        g.moe_few(x, r, gate, gate, down, 2)
