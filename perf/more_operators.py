"""The 8-bit products, the norm before them and the expert order around them as they are called, and their plain forms.

A case names one operator, its sizes, types and layouts.  ``own`` false computes
it with elementary torch operations in 32 bits; ``own`` true calls the package.

8 bits: 128 consecutive values along the contracted axis share a scale 2**s, s the
smallest exponent with largest magnitude <= 448 * 2**s, and each value is held as
the nearest e4m3 number (ties to the even code) times the scale.
"""
import math

import torch

own = False

BLOCK = 128
EPS = 1e-6
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # the norm before a projection in a decode step of 16 tokens: the smallest call, its latency counts
        {"name": "norm_16x8192", "op": "norm", "rows": 16, "d": 8192, "dtype": "f16", "residual": True, "quantize": True},
        # rows that start anywhere, the norm's output in the type of its input
        {"name": "norm_3001x4097", "op": "norm", "rows": 3001, "d": 4097, "dtype": "bf16", "residual": True,
         "quantize": False},
        # a prefill batch, the output in 8 bits for the product that follows
        {"name": "norm_131072x7168", "op": "norm", "rows": 131072, "d": 7168, "dtype": "f16", "residual": True,
         "quantize": True},
        # a decode step of 16 tokens through an output projection, activations quantised within the call
        {"name": "mm_16x16384x8192", "op": "mm", "m": 16, "n": 16384, "k": 8192, "dtype": "f16", "held": False,
         "bias": False, "act": "none"},
        # no dimension a tile or a block divides, with the fused output stage
        {"name": "mm_3001x1999x4097", "op": "mm", "m": 3001, "n": 1999, "k": 4097, "dtype": "bf16", "held": False,
         "bias": True, "act": "gelu"},
        # the routed rows of a prefill batch times one weight, both held in 8 bits
        {"name": "mm_131072x2048x7168", "op": "mm", "m": 131072, "n": 2048, "k": 7168, "dtype": "f16", "held": True,
         "bias": False, "act": "none"},
        # 64 tokens of 8 choices over 64 experts, gate and up: a stream of weights
        {"name": "grouped_512_g64_2048x7168_up", "op": "grouped", "rows": 512, "groups": 64, "n": 2048, "k": 7168,
         "skew": 0.5, "dtype": "f16", "held": False, "gated": True},
        # the experts' second projection of a prefill batch, unevenly filled
        {"name": "grouped_131072_g8_7168x2048", "op": "grouped", "rows": 131072, "groups": 8, "n": 7168, "k": 2048,
         "skew": 0.7, "dtype": "bf16", "held": True, "gated": False},
        # 16 tokens put into their experts' order
        {"name": "gather_16x8_e64_7168", "op": "gather", "t": 16, "top": 8, "e": 64, "d": 7168, "dtype": "f16"},
        # a prefill batch put into its experts' order
        {"name": "gather_16384x8_e64_7168", "op": "gather", "t": 16384, "top": 8, "e": 64, "d": 7168, "dtype": "f16"},
        # and the experts' outputs back, weighted
        {"name": "combine_16384x8_e64_7168", "op": "combine", "t": 16384, "top": 8, "e": 64, "d": 7168, "dtype": "f16"},
        # the gradient of that, for the experts' outputs and for the weights
        {"name": "combine_grad_16384x8_e64_2048", "op": "combine_grad", "t": 16384, "top": 8, "e": 64, "d": 2048,
         "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi):
    """A size of the range, two in three of them multiples of 64."""
    return _log(rng, lo, hi) if rng.random() < 0.34 else 64 * _log(rng, max(1, lo // 64), hi // 64)


def draw(rng):
    op = rng.choice(("norm", "mm", "mm", "grouped", "grouped", "gather", "combine", "combine_grad"))
    dtype = rng.choice(sorted(DTYPES))
    if op == "norm":
        return {"op": op, "rows": _log(rng, 1, 65536), "d": _size(rng, 64, 12288), "dtype": dtype,
                "residual": rng.random() < 0.7, "quantize": rng.random() < 0.6}
    most = 131072 * 2048 * 7168
    if op == "mm":
        n, k = _size(rng, 16, 16384), _size(rng, 64, 8192)
        return {"op": op, "m": _log(rng, 1, min(65536, most // (n * k))), "n": n, "k": k, "dtype": dtype,
                "held": rng.random() < 0.5, "bias": rng.random() < 0.5,
                "act": rng.choice(("none", "relu", "silu", "gelu"))}
    if op == "grouped":
        gated = rng.random() < 0.5
        n, k = _size(rng, 64, 4096), _size(rng, 64, 8192)
        return {"op": op, "rows": _log(rng, 1, min(65536, most // (n * k * (2 if gated else 1)))),
                "groups": _log(rng, 1, 64), "n": n, "k": k, "skew": round(rng.uniform(0, 2), 2), "dtype": dtype,
                "held": rng.random() < 0.5, "gated": gated}
    e = _log(rng, 4, 256)
    return {"op": op, "t": _log(rng, 1, 16384), "top": rng.randint(1, min(8, e)), "e": e, "d": _size(rng, 64, 7168),
            "dtype": dtype}


# ------------------------------------------------------------------ inputs
def _normal(gen, *shape, dtype=torch.float16, scale=1.0):
    v = torch.empty(shape, dtype=dtype, device="cuda")
    return v.normal_(0.0, scale, generator=gen)


def _kept(w):
    """A weight [.., contracted, columns] as the program keeps it in 8 bits."""
    if own:
        import dense_tiled_gemm_fp16_gb300 as g
        return g.fp8_quantize(w, axis=-2)
    return _to_fp8(w.transpose(-1, -2))


def _activations(x, held):
    if not held:
        return x
    if own:
        import dense_tiled_gemm_fp16_gb300 as g
        return g.fp8_quantize(x)
    return _to_fp8(x)


def _weight(gen, c, *lead):
    """A weight stored with the contracted axis last, seen as [.., k, n]."""
    return _normal(gen, *lead, c["n"], c["k"], dtype=DTYPES[c["dtype"]], scale=c["k"] ** -0.5).transpose(-1, -2)


def _group_rows(gen, c):
    """Rows of each group: every row takes a group, the groups unevenly likely (an empty one may come up)."""
    p = torch.exp(c["skew"] * _normal(gen, c["groups"], dtype=torch.float32))
    at = torch.multinomial(p, c["rows"], replacement=True, generator=gen)
    return torch.bincount(at, minlength=c["groups"]).int()


def _choices(gen, c):
    """Distinct experts of each token, the experts unevenly liked."""
    like = 0.5 * _normal(gen, c["e"], dtype=torch.float32)
    v = like + _normal(gen, c["t"], c["e"], dtype=torch.float32)
    return torch.sort(v, dim=1, descending=True, stable=True).indices[:, :c["top"]].int().contiguous()


def _order(ids, e):
    """(place of each choice in its experts' order, choice at each place, choices of each expert)."""
    flat = ids.flatten().long()
    order = torch.sort(flat, stable=True).indices
    rows = torch.empty_like(order)
    rows[order] = torch.arange(order.numel(), device=order.device)
    return rows.view(ids.shape).int(), order.int(), torch.bincount(flat, minlength=e).int()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    c, s, dt = case, {"case": case}, DTYPES[case["dtype"]]
    if c["op"] == "norm":
        s["x"] = _normal(gen, c["rows"], c["d"], dtype=dt)
        s["residual"] = _normal(gen, c["rows"], c["d"], dtype=dt, scale=3.0) if c["residual"] else None
        s["weight"] = 1 + _normal(gen, c["d"], dtype=dt, scale=0.2)
    elif c["op"] == "mm":
        s["a"] = _activations(_normal(gen, c["m"], c["k"], dtype=dt), c["held"])
        s["b"] = _kept(_weight(gen, c))
        s["bias"] = _normal(gen, c["n"], dtype=dt) if c["bias"] else None
    elif c["op"] == "grouped":
        s["a"] = _activations(_normal(gen, c["rows"], c["k"], dtype=dt), c["held"])
        s["b"] = _kept(_weight(gen, c, c["groups"]))
        s["b_up"] = _kept(_weight(gen, c, c["groups"])) if c["gated"] else None
        s["group_rows"] = _group_rows(gen, c)
    else:
        s["ids"] = _choices(gen, c)
        s["order"] = _order(s["ids"], c["e"])  # what the program keeps from the way there for the way back
        if c["op"] == "gather":
            s["x"] = _normal(gen, c["t"], c["d"], dtype=dt)
        else:
            s["y"] = _normal(gen, c["t"] * c["top"], c["d"], dtype=dt)
            w = torch.exp(_normal(gen, c["t"], c["top"], dtype=torch.float32))
            s["weights"] = w / w.sum(dim=1, keepdim=True)
        if c["op"] == "combine_grad":
            s["dy"] = _normal(gen, c["t"], c["d"], dtype=dt)
    return s


# ------------------------------------------------------------------ plain forms
def _pow2(e):
    """2**e exactly, e from -126 to 127."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _to_fp8(x):
    """(e4m3 values [.., blocks, 128], scale exponents [.., blocks, 1], k) along the last axis."""
    k = x.shape[-1]
    v = torch.nn.functional.pad(x.float(), (0, -k % BLOCK)).unflatten(-1, (-1, BLOCK))
    m, e = torch.frexp(v.abs().amax(dim=-1, keepdim=True))  # m in [0.5, 1): 448 is 0.875 * 2**9
    s = torch.where(m > 0, torch.where(m <= 0.875, e - 9, e - 8), -126).clamp(-126, 126)
    return (v * _pow2(-s)).to(torch.float8_e4m3fn), s.to(torch.int8), k


def _from_fp8(q):
    """The values in 32 bits."""
    v, s, k = q
    return (v.float() * _pow2(s)).flatten(-2)[..., :k]


def _act(name, v):
    if name == "relu":
        return v.clamp_min(0)
    if name == "silu":
        return v / (1 + torch.exp(-v))
    if name == "gelu":
        return 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    return v


def _plain_norm(s):
    c, x = s["case"], s["x"]
    h = x if s["residual"] is None else (x.float() + s["residual"].float()).to(x.dtype)
    v = h.float()
    y = v * (1 / torch.sqrt((v * v).mean(dim=1, keepdim=True) + EPS)) * s["weight"].float()
    y = (_from_fp8(_to_fp8(y)) if c["quantize"] else y).to(x.dtype)
    return {"y": y} if s["residual"] is None else {"y": y, "sum": h}


def _in_8_bits(a):
    return _from_fp8(a if isinstance(a, tuple) else _to_fp8(a))


def _plain_mm(s):
    c = s["case"]
    v = _in_8_bits(s["a"]) @ _from_fp8(s["b"]).t()
    if s["bias"] is not None:
        v = v + s["bias"].float()
    return _act(c["act"], v).to(DTYPES[c["dtype"]])


def _of_group(q, g):
    return _from_fp8((q[0][g], q[1][g], q[2])).t()


def _plain_grouped(s):
    c, a = s["case"], _in_8_bits(s["a"])
    parts = []
    for g, v in enumerate(a.split(s["group_rows"].tolist())):
        y = v @ _of_group(s["b"], g)
        parts.append((_act("silu", y) * (v @ _of_group(s["b_up"], g)) if c["gated"] else y).to(DTYPES[c["dtype"]]))
    return torch.cat(parts)


def _plain_gather(s):
    rows, order, group_rows = _order(s["ids"], s["case"]["e"])
    return {"x": s["x"][order.long() // s["case"]["top"]], "rows": rows, "order": order, "group_rows": group_rows}


def _plain_combine(s):
    v = s["y"][s["order"][0].long()].float()
    return (s["weights"].unsqueeze(2) * v).sum(dim=1).to(s["y"].dtype)


def _plain_combine_grad(s):
    c, dy = s["case"], s["dy"].float()
    rows, order, _ = s["order"]
    dweights = (s["y"][rows.long()].float() * dy.unsqueeze(1)).sum(dim=2)
    at = order.long()
    return {"dy": (s["weights"].flatten()[at].unsqueeze(1) * dy[at // c["top"]]).to(s["y"].dtype), "dweights": dweights}


def _own(s):
    import dense_tiled_gemm_fp16_gb300 as g

    c = s["case"]
    if c["op"] == "norm":
        y = g.rms_norm(s["x"], s["weight"], eps=EPS, residual=s["residual"], quantize=c["quantize"])
        y, h = y if c["residual"] else (y, None)
        y = g.fp8_dequantize(y, dtype=s["x"].dtype) if c["quantize"] else y
        return {"y": y, "sum": h} if c["residual"] else {"y": y}
    if c["op"] == "mm":
        return g.fp8_mm(s["a"], s["b"], bias=s["bias"], act=c["act"], dtype=DTYPES[c["dtype"]])
    if c["op"] == "grouped":
        return g.fp8_grouped_mm(s["a"], s["b"], s["group_rows"], act="silu" if c["gated"] else "none", b_up=s["b_up"],
                                dtype=DTYPES[c["dtype"]])
    if c["op"] == "gather":
        order = g.moe_sort(s["ids"], c["e"])
        return {"x": g.moe_gather(s["x"], order), "rows": order.rows, "order": order.order,
                "group_rows": order.group_rows}
    order = g.MoeOrder(*s["order"])
    if c["op"] == "combine":
        return g.moe_combine(s["y"], order, s["weights"])
    dy, dweights = g.moe_combine_grad(s["dy"], s["y"], order, s["weights"])
    return {"dy": dy, "dweights": dweights}


def run(state):
    """One pass.  A norm's output in 8 bits goes back to the type of its input, so that it comes out as values."""
    if own:
        return _own(state)
    return {"norm": _plain_norm, "mm": _plain_mm, "grouped": _plain_grouped, "gather": _plain_gather,
            "combine": _plain_combine, "combine_grad": _plain_combine_grad}[state["case"]["op"]](state)


# ------------------------------------------------------------------ work
def _packed(rows, k):
    """Bytes of rows x k values in 8 bits with their scales."""
    return rows * (k + -(-k // BLOCK))


def work(case):
    c = case
    if c["op"] == "norm":
        n = c["rows"] * c["d"]
        out = _packed(c["rows"], c["d"]) + 2 * n if c["quantize"] else 2 * n
        return {"bytes": 2 * n + (4 * n if c["residual"] else 0) + 2 * c["d"] + out, "flops": 4 * n}
    if c["op"] in ("mm", "grouped"):
        m, n, k = c["m" if c["op"] == "mm" else "rows"], c["n"], c["k"]
        a = _packed(m, k) if c["held"] else 2 * m * k
        if c["op"] == "mm":
            return {"bytes": a + _packed(n, k) + 2 * m * n + (2 * n if c["bias"] else 0), "flops": 2 * m * n * k}
        both = 2 if c["gated"] else 1
        reached = c["groups"] * (1 - (1 - 1 / c["groups"]) ** m)  # of even groups: the expected number
        return {"bytes": a + reached * both * _packed(n, k) + 2 * m * n + 4 * c["groups"], "flops": 2 * m * n * k * both}
    r, n = c["t"] * c["top"], c["t"] * c["d"]
    if c["op"] == "gather":
        return {"bytes": 2 * n + 2 * r * c["d"] + 12 * r + 4 * c["e"], "flops": r}
    if c["op"] == "combine":
        return {"bytes": 2 * r * c["d"] + 2 * n + 8 * r, "flops": 2 * r * c["d"]}
    return {"bytes": 4 * r * c["d"] + 2 * n + 12 * r, "flops": 3 * r * c["d"]}


# ------------------------------------------------------------------ 64 bits, from the definition
def _grid64(x):
    """x along its last axis as 8 bits hold it, in 64 bits."""
    k = x.shape[-1]
    blocks = torch.nn.functional.pad(x.double(), (0, -k % BLOCK)).reshape(*x.shape[:-1], -1, BLOCK)
    big = blocks.abs().max(dim=-1, keepdim=True).values.clamp_min(2.0 ** -1000)
    s = torch.ceil(torch.log2(big / 448.0)).clamp(-126, 126)
    s = torch.where(big <= 448.0 * torch.exp2(s - 1), s - 1, s)  # (the logarithm's own error)
    s = torch.where(big > 448.0 * torch.exp2(s), s + 1, s).clamp(-126, 126)
    scale = ((s.long() + 1023) << 52).view(torch.float64)
    a = blocks / scale
    expo = (((a.abs().clamp_min(2.0 ** -6).view(torch.int64) >> 52) - 1023 - 3 + 1023) << 52).view(torch.float64)
    return (torch.round(a / expo) * expo * scale).flatten(-2)[..., :k]


def _act64(name, v):
    f = torch.nn.functional
    return {"none": lambda t: t, "relu": f.relu, "silu": f.silu, "gelu": f.gelu}[name](v)


def _exact_norm(c, seed):
    s = prepare(c, seed)
    h = s["x"] if s["residual"] is None else (s["x"].double() + s["residual"].double()).to(s["x"].dtype)
    parts = []
    for v in h.split(1 << 14):
        v = v.double()
        y = v * torch.rsqrt((v ** 2).sum(dim=1, keepdim=True) / c["d"] + EPS) * s["weight"].double()
        parts.append(_grid64(y) if c["quantize"] else y)
    y = torch.cat(parts)
    return {"y": y} if s["residual"] is None else {"y": y, "sum": h.double()}


def exact(case, seed):
    c = case
    if c["op"] == "norm":
        return _exact_norm(c, seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[c["dtype"]]
    if c["op"] == "mm":
        x = _normal(gen, c["m"], c["k"], dtype=dt)
        b = _grid64(_weight(gen, c).transpose(0, 1)).t()
        bias = _normal(gen, c["n"], dtype=dt) if c["bias"] else None
        v = torch.cat([_grid64(p) @ b for p in x.split(1 << 14)])
        return _act64(c["act"], v if bias is None else v + bias.double())
    if c["op"] == "grouped":
        x = _normal(gen, c["rows"], c["k"], dtype=dt)
        ws = [_weight(gen, c, c["groups"]) for _ in range(2 if c["gated"] else 1)]
        ends = _group_rows(gen, c).cumsum(0).tolist()
        y = torch.zeros(c["rows"], c["n"], dtype=torch.float64, device="cuda")
        for g, hi in enumerate(ends):
            lo = ends[g - 1] if g else 0
            mats = [_grid64(w[g].t()).t() for w in ws] if hi > lo else []
            for i in range(lo, hi, 1 << 14):
                v = _grid64(x[i:min(hi, i + (1 << 14))])
                p = [v @ m for m in mats]
                y[i:min(hi, i + (1 << 14))] = _act64("silu", p[0]) * p[1] if c["gated"] else p[0]
        return y
    s = prepare(c, seed)
    key = s["ids"].long().flatten() * s["ids"].numel() + torch.arange(s["ids"].numel(), device="cuda")
    order = torch.argsort(key)  # by expert, then by the choice's own number
    rows = torch.argsort(order).view(s["ids"].shape)
    if c["op"] == "gather":
        counts = (s["ids"].flatten()[:, None] == torch.arange(c["e"], device="cuda")).sum(dim=0)
        return {"x": s["x"].index_select(0, order // c["top"]).double(), "rows": rows.int(), "order": order.int(),
                "group_rows": counts.int()}
    w = s["weights"].double()
    if c["op"] == "combine":
        y = torch.zeros(c["t"], c["d"], dtype=torch.float64, device="cuda")
        for j in range(c["top"]):
            y.addcmul_(w[:, j:j + 1], s["y"][rows[:, j]].double())
        return y
    dys = torch.zeros(c["t"] * c["top"], c["d"], dtype=torch.float64, device="cuda")
    dw, dy = torch.zeros_like(w), s["dy"].double()
    for j in range(c["top"]):
        dys[rows[:, j]] = w[:, j:j + 1] * dy
        dw[:, j] = torch.einsum("td,td->t", s["y"][rows[:, j]].double(), dy)
    return {"dy": dys, "dweights": dw}
