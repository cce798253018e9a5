"""The MXFP4 and few-token mixture-of-experts operators as they are called, and their plain forms.

A case names one operator, its sizes, types and layouts.  ``own`` false computes
it with elementary torch operations in 32 bits; ``own`` true calls the package.

MXFP4: 32 consecutive values along the contracted axis share a scale 2**s with
s = floor(log2(largest magnitude)) - 2, and each value is held as the nearest of
0, 0.5, 1, 1.5, 2, 3, 4, 6 (ties to the even code) times the scale, with its sign.
"""
import math

import torch

own = False

BLOCK = 32
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # the activations of one decode step of 16 tokens
        {"name": "quantize_16x8192", "op": "quantize", "rows": 16, "k": 8192, "dtype": "f16", "transposed": False},
        # an irregular operand read through its transpose, neither size a multiple of a block
        {"name": "quantize_3001x4097_t", "op": "quantize", "rows": 3001, "k": 4097, "dtype": "bf16", "transposed": True},
        # the routed rows of a prefill batch through a mixture-of-experts layer
        {"name": "quantize_131072x7168", "op": "quantize", "rows": 131072, "k": 7168, "dtype": "f16",
         "transposed": False},
        # one token through an output projection: the smallest product, the launch and the weight stream
        {"name": "mm_1x16384x8192", "op": "mm", "m": 1, "n": 16384, "k": 8192, "a": "f16", "bias": False, "act": "none"},
        # a decode step of 16 tokens, activations quantised within the call
        {"name": "mm_16x16384x8192", "op": "mm", "m": 16, "n": 16384, "k": 8192, "a": "f16", "bias": True, "act": "none"},
        # no dimension a tile divides, with the fused output stage
        {"name": "mm_3001x1999x4097", "op": "mm", "m": 3001, "n": 1999, "k": 4097, "a": "f16", "bias": True,
         "act": "gelu"},
        # a square product of two operands that are held in 4 bits
        {"name": "mm_4096", "op": "mm", "m": 4096, "n": 4096, "k": 4096, "a": "mxf4", "bias": False, "act": "none"},
        # the routed rows of a prefill batch times one weight, both held in 4 bits
        {"name": "mm_131072x2048x7168", "op": "mm", "m": 131072, "n": 2048, "k": 7168, "a": "mxf4", "bias": False,
         "act": "none"},
        # one token through a layer of 8 wide experts in fp16, weights stored with the contracted axis last
        {"name": "moe_1_e8_7168", "op": "moe", "t": 1, "e": 8, "d": 7168, "f": 2048, "top": 4, "weights": "f16",
         "order": "nk", "renormalize": True, "act": "silu"},
        # 16 tokens over many narrow experts in fp16, weights stored row-major [d, f]
        {"name": "moe_16_e64_2048", "op": "moe", "t": 16, "e": 64, "d": 2048, "f": 1024, "top": 8, "weights": "f16",
         "order": "kn", "renormalize": True, "act": "silu"},
        # 4 tokens over many experts held in 4 bits
        {"name": "moe_4_e64_2048_mxf4", "op": "moe", "t": 4, "e": 64, "d": 2048, "f": 1024, "top": 8,
         "weights": "mxf4", "order": "nk", "renormalize": False, "act": "silu"},
        # the largest call of the layer: 64 tokens, every expert reached, weights in 4 bits
        {"name": "moe_64_e64_7168_mxf4", "op": "moe", "t": 64, "e": 64, "d": 7168, "f": 2048, "top": 8,
         "weights": "mxf4", "order": "nk", "renormalize": True, "act": "silu"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("quantize", "mm", "mm", "moe", "moe"))
    if op == "quantize":
        return {"op": op, "rows": _log(rng, 1, 65536), "k": _log(rng, 8, 12288), "dtype": rng.choice(sorted(DTYPES)),
                "transposed": rng.random() < 0.3}
    if op == "mm":
        return {"op": op, "m": _log(rng, 1, 65536), "n": _log(rng, 16, 16384), "k": _log(rng, 64, 8192),
                "a": rng.choice(("f16", "mxf4")), "bias": rng.random() < 0.5,
                "act": rng.choice(("none", "relu", "silu", "gelu"))}
    e = _log(rng, 4, 64)
    odd = rng.random() < 0.2  # sizes that no vector divides
    size = (lambda lo, hi: _log(rng, lo, hi)) if odd else (lambda lo, hi: 64 * _log(rng, lo / 64, hi / 64))
    return {"op": op, "t": _log(rng, 1, 64), "e": e, "d": size(256, 7168), "f": size(128, 2048),
            "top": rng.randint(1, min(8, e)), "weights": rng.choice(("f16", "mxf4")), "order": rng.choice(("nk", "kn")),
            "renormalize": rng.random() < 0.7, "act": rng.choice(("silu", "gelu"))}


# ------------------------------------------------------------------ inputs
def _normal(gen, *shape, dtype=torch.float16, scale=1.0):
    v = torch.empty(shape, dtype=dtype, device="cuda")
    return v.normal_(0.0, scale, generator=gen)


def _tokens(gen, case, w_router):
    """Tokens whose choice of experts does not hang on the last bits of a sum: the gap between the last
    expert taken and the first one left is over 1e-4 (logits have a deviation of 1)."""
    t, top = case["t"], case["top"]
    x = _normal(gen, 2 * t + 8, case["d"])
    v = (x.double() @ w_router.double()).sort(dim=1, descending=True).values
    steps = v[:, :-1] - v[:, 1:]  # the order among the chosen counts too: it is the order of the output
    hard = (steps[:, :top] < 1e-4).any(dim=1)
    return x[torch.sort(hard.int(), stable=True).indices[:t]].contiguous()


def _weight(gen, case, rows, cols):
    """Expert weights [e, rows, cols], rows contracted, stored in the case's order."""
    e, scale = case["e"], rows ** -0.5
    if case["order"] == "nk":
        return _normal(gen, e, cols, rows, scale=scale).transpose(1, 2)
    return _normal(gen, e, rows, cols, scale=scale)


def _kept(w, axis):
    """A weight as the program keeps it in 4 bits."""
    if own:
        import dense_tiled_gemm_fp16_gb300 as g
        return g.mxf4_quantize(w, axis=axis)
    return _to_mxf4(w.movedim(axis, -1))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    if case["op"] == "quantize":
        dt = DTYPES[case["dtype"]]
        if case["transposed"]:
            x = _normal(gen, case["k"], case["rows"], dtype=dt).t()
        else:
            x = _normal(gen, case["rows"], case["k"], dtype=dt)
        s["x"] = x
    elif case["op"] == "mm":
        x = _normal(gen, case["m"], case["k"])
        w = _normal(gen, case["n"], case["k"], scale=case["k"] ** -0.5)
        s["bias"] = _normal(gen, case["n"]) if case["bias"] else None
        s["a"] = x if case["a"] == "f16" else _kept(x, -1)
        s["b"] = _kept(w, -1)
    else:
        s["router"] = _normal(gen, case["d"], case["e"], scale=case["d"] ** -0.5)
        s["x"] = _tokens(gen, case, s["router"])
        for name, rows, cols in (("gate", "d", "f"), ("up", "d", "f"), ("down", "f", "d")):
            w = _weight(gen, case, case[rows], case[cols])
            s[name] = w if case["weights"] == "f16" else _kept(w, -2)
    return s


# ------------------------------------------------------------------ plain forms
def _pow2(e):
    """2**e exactly, e from -252 to 127 (torch.ldexp goes by a power that may be an ulp off)."""
    normal = ((e.int().clamp_min(-126) + 127) << 23).view(torch.float32)
    return normal * (((e.int() + 126).clamp_max(0) + 127) << 23).view(torch.float32)


def _to_mxf4(x):
    """(twice the e2m1 values as int8 [..., k], scale exponents as int16 [..., blocks], k) along the last axis."""
    k = x.shape[-1]
    v = torch.nn.functional.pad(x.float(), (0, -k % BLOCK)).unflatten(-1, (-1, BLOCK))
    top = v.abs().amax(dim=-1)
    s = torch.where(top > 0, (torch.frexp(top).exponent - 3).clamp(-127, 127), -127)
    v = (v * _pow2(-s).unsqueeze(-1)).clamp(-6.0, 6.0)
    a = v.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    twice = (torch.round(v / step) * step * 2).to(torch.int8)
    return twice.flatten(-2)[..., :k].contiguous(), s.to(torch.int16), k


def _from_mxf4(q):
    """The values in 32 bits."""
    twice, s, k = q
    v = torch.nn.functional.pad(twice.float(), (0, -k % BLOCK)).unflatten(-1, (-1, BLOCK))
    return (v * _pow2(s - 1).unsqueeze(-1)).flatten(-2)[..., :k]


def _act(name, v):
    if name == "relu":
        return v.clamp_min(0)
    if name == "silu":
        return v / (1 + torch.exp(-v))
    if name == "gelu":
        return 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    return v


def _plain_mm(s):
    c = s["case"]
    a = _from_mxf4(_to_mxf4(s["a"]) if c["a"] == "f16" else s["a"])
    v = a @ _from_mxf4(s["b"]).t()
    if s["bias"] is not None:
        v = v + s["bias"].float()
    return _act(c["act"], v).half()


def _plain_moe(s):
    c, x = s["case"], s["x"].float()
    t, top = c["t"], c["top"]
    logits = x @ s["router"].float()
    best, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    best, ids = best[:, :top], ids[:, :top]
    z = torch.exp(best - best[:, :1])
    total = z.sum(dim=1, keepdim=True) if c["renormalize"] else torch.exp(logits - best[:, :1]).sum(dim=1, keepdim=True)
    w = z / total
    few = t * top <= c["e"]  # fewer choices than experts: only the chosen weights are looked at

    def weight(name):  # [experts or choices, contracted, columns]
        m = s[name]
        if c["weights"] == "mxf4":
            m = (m[0][ids.flatten()], m[1][ids.flatten()], m[2]) if few else m
            return _from_mxf4(m).transpose(1, 2)
        return (m[ids.flatten()] if few else m).float()

    v = x.repeat_interleave(top, dim=0).unsqueeze(1) if few else x.expand(c["e"], t, c["d"])
    h = _act(c["act"], torch.bmm(v, weight("gate"))) * torch.bmm(v, weight("up"))
    y = torch.bmm(h, weight("down"))
    y = y.view(t, top, c["d"]) if few else y[ids, torch.arange(t, device=x.device).unsqueeze(1)]
    return {"y": (w.unsqueeze(2) * y).sum(dim=1).half(), "weights": w, "ids": ids.int()}


def _own(s):
    import dense_tiled_gemm_fp16_gb300 as g

    c = s["case"]
    if c["op"] == "quantize":
        return g.mxf4_dequantize(g.mxf4_quantize(s["x"]))
    if c["op"] == "mm":
        return g.mxf4_mm(s["a"], s["b"], bias=s["bias"], act=c["act"])
    y, weights, ids = g.moe_few(s["x"], s["router"], s["gate"], s["up"], s["down"], c["top"], act=c["act"],
                                renormalize=c["renormalize"])
    return {"y": y, "weights": weights, "ids": ids}


def run(state):
    """One pass.  "quantize" is to 4 bits and back to fp16, so that what is held in 4 bits comes out as values."""
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "quantize":
        return _from_mxf4(_to_mxf4(state["x"])).half()
    return _plain_mm(state) if op == "mm" else _plain_moe(state)


# ------------------------------------------------------------------ work
def _packed(rows, k):
    """Bytes of rows x k values in 4 bits with their scales."""
    return rows * (k / 2 + -(-k // BLOCK))


def _reached(t, e, top):
    """Experts that t tokens reach, each choosing `top` of e evenly: the expected number."""
    return e * (1 - (1 - top / e) ** t)


def work(case):
    c = case
    if c["op"] == "quantize":
        n = c["rows"] * c["k"]
        return {"bytes": n * DTYPES[c["dtype"]].itemsize + _packed(c["rows"], c["k"]) + 2 * n, "flops": 4 * n}
    if c["op"] == "mm":
        m, n, k = c["m"], c["n"], c["k"]
        a = 2 * m * k if c["a"] == "f16" else _packed(m, k)
        return {"bytes": a + _packed(n, k) + 2 * m * n + (2 * n if c["bias"] else 0), "flops": 2 * m * n * k}
    t, e, d, f, top = c["t"], c["e"], c["d"], c["f"], c["top"]
    one = 6 * d * f if c["weights"] == "f16" else 2 * _packed(f, d) + _packed(d, f)
    return {"bytes": _reached(t, e, top) * one + 2 * d * e + 4 * t * d + 8 * t * top,
            "flops": 2 * t * d * e + 6 * t * top * d * f}


# ------------------------------------------------------------------ 64 bits, from the definition
def _grid64(x):
    """x along its last axis as MXFP4 holds it, in 64 bits: thresholds between neighbouring values, a value on
    one going to the even code."""
    k = x.shape[-1]
    blocks = torch.nn.functional.pad(x.double(), (0, -k % BLOCK)).reshape(*x.shape[:-1], -1, BLOCK)
    big = blocks.abs().max(dim=-1, keepdim=True).values.clamp_min(2.0 ** -1000)
    expo = (big.view(torch.int64) >> 52) - 1023  # of a normal number in 64 bits
    scale = (((expo - 2).clamp(-127, 127) + 1023) << 52).view(torch.float64)
    a = blocks.abs() / scale
    out = torch.zeros_like(a)
    for low, high, even_low in ((0.0, 0.5, True), (0.5, 1.0, False), (1.0, 1.5, True), (1.5, 2.0, False),
                                (2.0, 3.0, True), (3.0, 4.0, False), (4.0, 6.0, True)):
        mid = (low + high) / 2
        out = torch.where((a > mid) if even_low else (a >= mid), high, out)
    return (torch.sign(blocks) * out * scale).flatten(-2)[..., :k]


def _source(case, seed):
    """The case's inputs before anything is quantised."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = _normal(gen, case["m"], case["k"])
    w = _normal(gen, case["n"], case["k"], scale=case["k"] ** -0.5)
    return x, w, _normal(gen, case["n"]) if case["bias"] else None


def exact(case, seed):
    c = case
    if c["op"] == "quantize":
        x = prepare(c, seed)["x"]
        return torch.cat([_grid64(p) for p in x.split(1 << 14)])
    if c["op"] == "mm":
        x, w, bias = _source(c, seed)
        b = _grid64(w).t()
        v = torch.cat([_grid64(p) @ b for p in x.split(1 << 14)])
        return _act64(c["act"], v if bias is None else v + bias.double())
    gen = torch.Generator(device="cuda").manual_seed(seed)
    router = _normal(gen, c["d"], c["e"], scale=c["d"] ** -0.5)
    x = _tokens(gen, c, router).double()
    gate, up, down = (_weight(gen, c, c[r], c[q]) for r, q in (("d", "f"), ("d", "f"), ("f", "d")))
    logits = x @ router.double()
    p = torch.softmax(logits, dim=1)
    ids = torch.argsort(-logits, dim=1, stable=True)[:, :c["top"]]
    w = torch.gather(p, 1, ids)
    w = w / w.sum(dim=1, keepdim=True) if c["renormalize"] else w
    y = torch.zeros_like(x)
    for e in range(c["e"]):
        at, j = torch.nonzero(ids == e, as_tuple=True)
        if at.numel():
            g, u, d = ((m[e].double() if c["weights"] == "f16" else _grid64(m[e].t()).t()) for m in (gate, up, down))
            h = _act64(c["act"], x[at] @ g) * (x[at] @ u)
            y[at] += w[at, j].unsqueeze(1) * (h @ d)
    return {"y": y, "weights": w, "ids": ids.int()}


def _act64(name, v):
    f = torch.nn.functional
    return {"none": lambda t: t, "relu": f.relu, "silu": f.silu, "gelu": f.gelu}[name](v)
