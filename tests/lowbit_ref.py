"""The block-scaled formats in 64 bits, in plain numpy: what the low-bit operators' tests compare with."""
import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1])


def nearest(v, grid):
    """Index of the grid's number nearest to v >= 0, ties to the even index, larger ones to the last."""
    mid = (grid[1:] + grid[:-1]) / 2
    up = np.searchsorted(mid, v, side="left")  # midpoints below v
    tie = (up < mid.size) & (v == mid[np.minimum(up, mid.size - 1)]) & (up % 2 == 1)
    return up + tie


def blocks(x, block):
    """x [rows, cols] as [rows, blocks, block], a last shorter block filled with zeros."""
    rows, cols = x.shape
    n = -(-cols // block)
    v = np.zeros((rows, n * block))
    v[:, :cols] = x
    return v.reshape(rows, n, block)


def pow2_scale(amax, most):
    """Exponent of the smallest power of two (-127 at least) whose `most`-fold holds amax (finite)."""
    e = np.full(amax.shape, -127)
    for k in range(-127, 128):
        e = np.where(amax > most * 2.0 ** k, k + 1, e)
    return e


def quantise(x, block, bits, factor=1.0):
    """(codes uint8 [rows, cols] one a value, scale bytes [rows, blocks]) of x, float64."""
    rows, cols = x.shape
    v = blocks(np.asarray(x, np.float64) / factor, block)
    bad = ~np.isfinite(v).all(-1)
    v = np.where(bad[..., None], 0.0, v)
    amax = np.abs(v).max(-1)
    grid = E2M1 if bits == 4 else E4M3
    if bits == 4 and block == 16:
        raw = nearest(np.minimum(amax / 6, 1e6), E4M3)
        s = E4M3[raw]
        raw = np.where(bad, 0x7F, raw)
    else:
        e = pow2_scale(amax, grid[-1])
        s, raw = 2.0 ** e.astype(np.float64), np.where(bad, 255, e + 127)
    q = nearest(np.abs(v) / np.where(s > 0, s, 1.0)[..., None], grid)
    q = np.where((s > 0)[..., None], q, 0)
    code = np.where(np.signbit(v) & ~((s == 0) | bad)[..., None], q + grid.size * (1 if bits == 4 else 0), q)
    if bits == 8:
        code = np.where(np.signbit(v) & ~bad[..., None], q | 0x80, q)
    return code.reshape(rows, -1)[:, :cols].astype(np.uint8), raw.astype(np.uint8)


def scale_value(raw, e8m0):
    raw = raw.astype(np.int64)
    if e8m0:
        return np.where(raw == 255, np.nan, 2.0 ** (raw - 127.0))
    a = raw & 0x7F
    v = np.where(a < 8, a * 2.0 ** -9, (8 + a % 8) * 2.0 ** (a // 8 - 10.0))
    return np.where(a == 0x7F, np.nan, np.where(raw >= 128, -v, v))


def values4(codes, raw, block):
    """Values of E2M1 codes (one a value) and scale bytes."""
    v = E2M1[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    return v * np.repeat(scale_value(raw, block == 32), block, 1)[:, :codes.shape[1]]


def values8(codes, raw, block):
    v = scale_value(codes, False)
    return v * np.repeat(scale_value(raw, True), block, 1)[:, :codes.shape[1]]


def pack(codes):
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)


def unpack(b):
    return np.stack([b & 15, b >> 4], -1).reshape(b.shape[0], -1)


def tile(raw, rows=None):
    """Scale bytes [rows, n] in the tensor cores' order, [row blocks, groups, 512]; one scale at a time."""
    rows, n = raw.shape
    G = -(-n // 4)
    out = np.zeros((-(-rows // 128), G, 512), np.uint8)
    for r in range(rows):
        for k in range(n):
            out[r // 128, k // 4, (r % 32) * 16 + (r // 32 % 4) * 4 + k % 4] = raw[r, k]
    return out


def untile(t, rows, n):
    r, k = np.arange(rows)[:, None], np.arange(n)[None, :]
    return t[r // 128, k // 4, (r % 32) * 16 + (r // 32 % 4) * 4 + k % 4]
