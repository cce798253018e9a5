"""A mixture-of-experts layer for a few tokens on CUDA torch tensors.

Mirrors ``include/moe_f16.h`` (``moe_f16``, ``moe_f16_workspace_size``) and adds
the tensor form ``moe_few``.  The workspace is a torch allocation of the call's
stream, so calls on different streams never share one.
"""
from __future__ import annotations

import ctypes

from .mxf4 import Mxf4Matrix, _empty, _pkg, _run, _stream, _torch

WEIGHT_F16, WEIGHT_MXF4 = 0, 1
MAX_TOKENS, MAX_EXPERTS, MAX_TOP_K, MAX_DIM = 64, 512, 8, 32768

# Every symbol include/moe_f16.h declares.
EXPORTED = ("moe_f16_workspace_size", "moe_f16")


class MoeWeight(ctypes.Structure):
    """moe_f16_weight."""
    _fields_ = [("format", ctypes.c_int), ("data", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("stride_e", ctypes.c_int64), ("stride_i", ctypes.c_int64), ("stride_o", ctypes.c_int64)]


def declare(L) -> None:
    """Argument types of the header's functions on the loaded library."""
    P, I64, I, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
    W = ctypes.POINTER(MoeWeight)
    L.moe_f16_workspace_size.argtypes = [I64, I64, I64, I64, I64, ctypes.POINTER(SZ)]
    L.moe_f16.argtypes = [P, I64, I64, P, I64, I64, W, W, W, I64, I64, I64, I64, I64, I, I, P, I64, P, P, P, SZ, P]
    for name in EXPORTED:
        getattr(L, name).restype = I


# ------------------------------------------------------------ C-ABI mirrors
def moe_f16_workspace_size(T: int, D: int, F: int, E: int, top_k: int) -> int:
    g = _pkg()
    n = ctypes.c_size_t(0)
    g._check(g.lib().moe_f16_workspace_size(T, D, F, E, top_k, ctypes.byref(n)), "moe_f16_workspace_size")
    return n.value


def moe_f16(x: int, stride_xt: int, stride_xi: int, router: int, stride_ri: int, stride_re: int, gate: MoeWeight,
            up: MoeWeight, down: MoeWeight, T: int, D: int, F: int, E: int, top_k: int, renormalize: int, act: int,
            y: int, ldy: int, weights: int, ids: int, workspace: int, workspace_bytes: int, stream: int = 0) -> None:
    """The layer on device pointers (see include/moe_f16.h)."""
    g = _pkg()
    g._check(g.lib().moe_f16(x, stride_xt, stride_xi, router, stride_ri, stride_re, gate, up, down, T, D, F, E, top_k,
                             renormalize, act, y, ldy, weights, ids, workspace, workspace_bytes, stream or None),
             "moe_f16")


# ------------------------------------------------------------ torch helper
def _weight(w, rows: int, cols: int, experts: int, name: str):
    """The MoeWeight of an fp16 tensor [E, rows, cols] or the Mxf4Matrix that
    mxf4_quantize(.., axis=-2) makes of one ([E, cols, rows])."""
    if isinstance(w, Mxf4Matrix):
        if w.shape != (experts, cols, rows):
            raise ValueError(f"{name} in MXFP4 must be quantised along its contracted axis: expected "
                             f"{(experts, cols, rows)}, got {w.shape}")
        return MoeWeight(WEIGHT_MXF4, w.codes_ptr, w.scales_ptr, 0, 0, 0)
    if w.dtype is not _torch().float16:
        raise TypeError("moe_few takes float16 tensors and Mxf4Matrix weights")
    if w.shape != (experts, rows, cols):
        raise ValueError(f"{name} must be [{experts}, {rows}, {cols}], got {tuple(w.shape)}")
    se, si, so = w.stride()
    # (a dimension of one element may carry any stride)
    return MoeWeight(WEIGHT_F16, w.data_ptr(), None, se if experts > 1 else 0, si if rows > 1 else 1,
                     so if cols > 1 else (rows + 7) // 8 * 8)


def moe_few(x, router, gate, up, down, top_k: int, act="silu", renormalize: bool = True, out=None, stream=None):
    """A mixture-of-experts layer for at most MAX_TOKENS tokens.

    x [T, D] and router [D, E] float16; gate and up [E, D, F] and down [E, F, D]
    all float16 (any positive strides) or all Mxf4Matrix, quantised along the
    contracted axis (``mxf4_quantize(w, axis=-2)``).  Returns (y [T, D] float16,
    routing weights [T, top_k] float32, expert ids [T, top_k] int32), the last
    two in order of falling router logits, equal logits in index order.  With
    `renormalize` a token's weights are the softmax over its chosen experts,
    otherwise over all."""
    g, t = _pkg(), _torch()
    if x.dim() != 2 or router.dim() != 2 or x.shape[1] != router.shape[0]:
        raise ValueError("moe_few takes x [T, D] and router [D, E]")
    T, D = x.shape
    E = router.shape[1]
    quantised = isinstance(gate, Mxf4Matrix)
    if isinstance(up, Mxf4Matrix) != quantised or isinstance(down, Mxf4Matrix) != quantised:
        raise TypeError("the three projections share one format")
    if len(gate.shape) != 3:
        raise ValueError("gate must be [E, D, F]")
    F = gate.shape[1] if quantised else gate.shape[2]
    code = g._act(act)
    wg, wu, wd = _weight(gate, D, F, E, "gate"), _weight(up, D, F, E, "up"), _weight(down, F, D, E, "down")
    if out is not None:
        g._check_out(out, (T, D), "[T, D]")
    for name, v in (("x", x), ("router", router), ("out", out)):
        if v is not None and v.dtype is not t.float16:
            raise TypeError(f"moe_few takes {name} as a float16 tensor")
    device = x.device
    if device.type != "cuda" or any(v is not None and v.device != device for v in (router, gate, up, down, out)):
        raise ValueError("tensors must share one CUDA device")
    need = moe_f16_workspace_size(T, D, F, E, top_k)
    y = _empty((T, D), t.float16, device, stream) if out is None else out
    probs = _empty((T, top_k), t.float32, device, stream)
    ids = _empty((T, top_k), t.int32, device, stream)
    space = _empty(need, t.uint8, device, stream)
    sxt, sxi = x.stride()
    sri, sre = router.stride()
    _run(device, "moe_f16", x.data_ptr(), sxt if T > 1 else D, sxi if D > 1 else 1, router.data_ptr(),
         sri if D > 1 else (E + 7) // 8 * 8, sre if E > 1 else (D + 7) // 8 * 8, wg, wu, wd, T, D, F, E, top_k,
         1 if renormalize else 0, code, y.data_ptr(), y.stride(0) if T > 1 else D, probs.data_ptr(), ids.data_ptr(),
         space.data_ptr(), need, _stream(device, stream))
    return y, probs, ids
