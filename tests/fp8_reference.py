"""The 8-bit format in 64 bits, from its definition: the tests' plain implementation."""
import numpy as np

# The e4m3 numbers of codes 0 .. 126 (127 is NaN): subnormals of 2^-9, then 8 a power of two from 2^-6 on.
GRID = np.array([c * 2.0 ** -9 if c < 8 else (8 + c % 8) * 2.0 ** (c // 8 - 10) for c in range(127)])


def quantize64(x):
    """(codes [rows, 128 * blocks], scale codes [rows, blocks]) of a float64 matrix."""
    rows, k = x.shape
    nb = -(-k // 128)
    p = np.zeros((rows, nb * 128))
    p[:, :k] = x
    p = p.reshape(rows, nb, 128)
    top = np.abs(p).max(-1)
    good = np.isfinite(top)
    s = np.full((rows, nb), -127)
    some = good & (top > 0)
    m, e = np.frexp(top[some])   # top = m 2^e, 1/2 <= m < 1; 448 = 0.875 * 2^9
    s[some] = np.clip(np.where(m <= 0.875, e - 9, e - 8), -127, 127)
    assert (top[some] <= 448 * np.exp2(s[some].astype(np.float64))).all()
    scales = np.where(good, s + 127, 255).astype(np.uint8)
    a = np.where(good[..., None], np.abs(p) / np.exp2(s.astype(np.float64))[..., None], 0.0)
    at = np.clip(np.searchsorted(GRID, a, side="right") - 1, 0, 126)   # the number at or below
    up = np.minimum(at + 1, 126)
    mid = (GRID[at] + GRID[up]) / 2
    codes = np.where((a > mid) | ((a == mid) & (at % 2 == 1)), up, at).astype(np.uint8)
    codes |= ((np.signbit(p) & good[..., None]).astype(np.uint8) << 7)
    return codes.reshape(rows, nb * 128), scales


def dequantize64(codes, scales):
    """The values (NaN for the NaN scale), padding included."""
    v = GRID[codes & 127] * np.where(codes & 128, -1.0, 1.0)
    s = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127))
    return v * np.repeat(s, 128, axis=1) + 0.0   # (no negative zeros)


def held64(x):
    """x (a torch tensor or array of two dimensions) as 8 bits hold it."""
    x = np.asarray(x.double().cpu().numpy() if hasattr(x, "double") else x, dtype=np.float64)
    return dequantize64(*quantize64(x))[:, :x.shape[1]]


def scales_plain(tiled, rows, k):
    """[rows, blocks] of one matrix's tiled scales, checking that the padding is zero."""
    nb = -(-k // 128)
    rt, kt = -(-rows // 128), -(-nb // 4)
    t = tiled.reshape(rt, kt, 32, 4, 4)   # tile row, tile column, row % 32, row % 128 / 32, block % 4
    full = t.transpose(0, 3, 2, 1, 4).reshape(rt * 128, kt * 4)
    assert not full[rows:].any() and not full[:, nb:].any()
    return full[:rows, :nb]


def codes_plain(codes, rows, k):
    """[rows, k] of one matrix's codes, checking that the padding is zero."""
    c = codes.reshape(rows, -(-k // 128) * 128)
    assert not c[:, k:].any()
    return c[:, :k]
