"""One decode step with 4-bit weights: a mixture-of-experts layer for a few
tokens, then an output projection.

    python examples/moe_decode.py [--tokens 4] [--dim 2048] [--hidden 1024] [--experts 64] [--top 8] [--vocab 16384]

The experts' projections and the output projection are quantised once to MXFP4,
as a serving program would at load time; a step then is one call of moe_few and
one of mxf4_mm, the activations quantised on the way.  Prints the step's time
with the weights in fp16 and in MXFP4, the bytes of either, and how far apart
the two steps' outputs are.
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import dense_tiled_gemm_fp16_gb300 as g  # noqa: E402


def weights(dim, hidden, experts, vocab, device):
    """Random fp16 weights in the layouts of the library's products: [K, N] row-major."""
    def rnd(*shape):
        return torch.empty(shape, dtype=torch.float16, device=device).normal_(0.0, shape[-2] ** -0.5)
    return {"router": rnd(dim, experts), "gate": rnd(experts, dim, hidden), "up": rnd(experts, dim, hidden),
            "down": rnd(experts, hidden, dim), "head": rnd(dim, vocab)}


def quantised(w):
    """The same with everything but the router in MXFP4 along the contracted axis."""
    return {name: v if name == "router" else g.mxf4_quantize(v, axis=-2) for name, v in w.items()}


def step(x, w, top):
    """(logits over the vocabulary, the experts each token went to)."""
    y, _, ids = g.moe_few(x, w["router"], w["gate"], w["up"], w["down"], top)
    head = w["head"]
    return (g.mxf4_mm(y, head) if isinstance(head, g.Mxf4Matrix) else g.matmul(y, head)), ids


def timed(f, steps=20):
    for _ in range(3):
        f()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    for _ in range(steps):
        f()
    b.record()
    torch.cuda.synchronize()
    return a.elapsed_time(b) / steps * 1e3


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, value in (("tokens", 4), ("dim", 2048), ("hidden", 1024), ("experts", 64), ("top", 8), ("vocab", 16384)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args(argv)
    device = torch.device("cuda:0")
    torch.manual_seed(0)
    w16 = weights(a.dim, a.hidden, a.experts, a.vocab, device)
    w4 = quantised(w16)
    x = torch.randn(a.tokens, a.dim, device=device).half()
    out = {}
    for name, w in (("fp16", w16), ("mxfp4", w4)):
        logits, ids = step(x, w, a.top)
        size = sum(v.nbytes if isinstance(v, g.Mxf4Matrix) else v.numel() * 2 for v in w.values())
        out[name] = logits, ids
        print(f"{name}: {size / 1e6:.0f} MB of weights, {timed(lambda: step(x, w, a.top)):.1f} us a step")
    apart = (out["mxfp4"][0].float() - out["fp16"][0].float()).norm() / out["fp16"][0].float().norm()
    print(f"logits apart by {apart.item():.3f} of their norm; the same experts: {torch.equal(out['fp16'][1], out['mxfp4'][1])}")
    return out


if __name__ == "__main__":
    main()
