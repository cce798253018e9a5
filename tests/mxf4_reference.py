"""MXFP4 in 64 bits, from its definition: the tests' plain implementation."""
import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quantize64(x):
    """(codes [rows, 32 * blocks] 0..15, scale codes [rows, blocks] 0..255) of a float64 matrix."""
    rows, k = x.shape
    nb = -(-k // 32)
    p = np.zeros((rows, nb * 32))
    p[:, :k] = x
    p = p.reshape(rows, nb, 32)
    codes = np.zeros((rows, nb, 32), dtype=np.uint8)
    scales = np.zeros((rows, nb), dtype=np.uint8)
    top = np.abs(p).max(-1)
    good = np.isfinite(top)
    e = np.full((rows, nb), -127)
    some = good & (top > 0)
    e[some] = np.clip(np.frexp(top[some])[1] - 1 - 2, -127, 127)   # frexp: top = m 2^e, 1/2 <= m < 1
    scales[:] = np.where(good, e + 127, 255)
    a = np.abs(p) / np.exp2(e.astype(np.float64))[..., None]
    a = np.where(good[..., None], a, 0.0)
    # nearest: count the midpoints passed; a value on one goes up only to an even code
    for i in range(7):
        mid = (GRID[i] + GRID[i + 1]) / 2
        codes += ((a > mid) | ((a == mid) & (i % 2 == 1))).astype(np.uint8)
    codes |= (np.signbit(p) & (codes >= 0) & good[..., None]).astype(np.uint8) << 3
    return codes.reshape(rows, nb * 32), scales


def dequantize64(codes, scales):
    """The values (NaN for the NaN scale), padding included."""
    v = GRID[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    s = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127))
    return v * np.repeat(s, 32, axis=1) + 0.0   # (no negative zeros)


def scales_plain(tiled, rows, k):
    """[rows, blocks] of one matrix's tiled scales, checking that the padding is zero."""
    nb = -(-k // 32)
    rt, kt = -(-rows // 128), -(-nb // 4)
    t = tiled.reshape(rt, kt, 32, 4, 4)   # tile row, tile column, row % 32, row % 128 / 32, block % 4
    full = t.transpose(0, 3, 2, 1, 4).reshape(rt * 128, kt * 4)
    assert not full[rows:].any() and not full[:, nb:].any()
    return full[:rows, :nb]
