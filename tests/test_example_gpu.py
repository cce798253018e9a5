"""The decode example runs and its two forms agree as far as 4 bits allow."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_decode_step(capsys):
    spec = importlib.util.spec_from_file_location("moe_decode", os.path.join(ROOT, "examples", "moe_decode.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    out = m.main(["--tokens", "3", "--dim", "512", "--hidden", "256", "--experts", "16", "--top", "4", "--vocab", "1000"])
    (a, ia), (b, ib) = out["fp16"], out["mxfp4"]
    assert a.shape == b.shape == (3, 1000) and torch.equal(ia, ib)
    # an e2m1 value is off by up to a quarter of itself, some 0.1 in the root mean square; three
    # products in a row, the first two multiplied, leave a relative error well under one half
    assert (a.float() - b.float()).norm() < 0.5 * a.float().norm()
    assert "us a step" in capsys.readouterr().out
