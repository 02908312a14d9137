"""The 4-bit floating point formats in plain numpy, from their definition in the
header: values, rounding by comparison with every magnitude, scale bytes and the
scale layout.  Shares nothing with the library."""
import numpy as np

GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], np.float64)
BLOCK = {"mx": 32, "nv": 16}


def e4m3_table():
    b = np.arange(256)
    s, e, m = b >> 7, (b >> 3) & 15, b & 7
    v = np.where(e == 0, m / 8.0 * 2.0 ** -6, (1 + m / 8.0) * 2.0 ** (e - 7.0))
    v = np.where((e == 15) & (m == 7), np.nan, v)
    return np.where(s == 1, -v, v)


E4M3 = e4m3_table()


def nearest(a, grid):
    """Index of the value of an ascending grid nearest to a >= 0; ties to the even index."""
    i = np.clip(np.searchsorted(grid, a) - 1, 0, len(grid) - 2)
    lo, hi = a - grid[i], grid[i + 1] - a
    up = (hi < lo) | ((hi == lo) & (i % 2 == 1))
    return np.where(a >= grid[-1], len(grid) - 1, i + up)


def quantize(x, fmt, g=None):
    """f32 rows [n, K] -> (codes uint8 [n, K/2], scale bytes [n, K/block], values f32 [n, K])."""
    x = np.asarray(x, np.float32)
    n, K = x.shape
    b = x.reshape(n, K // BLOCK[fmt], BLOCK[fmt])
    with np.errstate(all="ignore"):
        m = np.abs(b).max(2)
        bad = ~np.isfinite(b).all(2)
        m = np.where(bad, 0, m).astype(np.float32)
        if fmt == "mx":
            byte = np.where(m > 0, np.clip(np.frexp(m.astype(np.float64))[1] - 1 - 2 + 127, 0, 254), 0)
            d = np.ldexp(1.0, byte - 127)
            q = b.astype(np.float64) / d[..., None]        # a power of two: exact
            byte = np.where(bad, 255, byte)
        else:
            g = np.float32(1.0 if g is None else g)
            t = m / (np.float32(6) * g)
            byte = nearest(np.minimum(t, np.float32(448)).astype(np.float64), E4M3[:127])
            d = E4M3[byte].astype(np.float32) * g
            r = np.where(d > 0, np.float32(1) / np.where(d > 0, d, 1), 0).astype(np.float32)
            q = (b * r[..., None]).astype(np.float32).astype(np.float64)
            byte = np.where(bad, 0x7F, byte)
        code = nearest(np.where(bad[..., None], 0, np.abs(q)), GRID)
        sign = np.signbit(b) & ~bad[..., None]
        if fmt == "nv":
            code = np.where(d[..., None] > 0, code, 0)
            sign = sign & (d[..., None] > 0)
        val = np.float32(GRID[code]) * np.float32(d)[..., None]
        val = np.where(bad[..., None], np.float32(np.nan), np.where(sign, -val, val))
    nib = (code + 8 * sign).astype(np.uint8).reshape(n, K)
    return (nib[:, 0::2] | nib[:, 1::2] << 4).astype(np.uint8), byte.astype(np.uint8), val.reshape(n, K).astype(np.float32)


def tile_scales(byte):
    """Scale bytes [rows, blocks] -> the header's layout (bytes past the matrix 0)."""
    rows, nb = byte.shape
    C = -(-nb // 4)
    out = np.zeros(-(-rows // 128) * C * 512, np.uint8)
    r, b = np.meshgrid(np.arange(rows), np.arange(nb), indexing="ij")
    out[((r // 128 * C + b // 4) * 32 + r % 32) * 16 + r % 128 // 32 * 4 + b % 4] = byte
    return out


def untile_scales(tiled, rows, nb):
    C = -(-nb // 4)
    r, b = np.meshgrid(np.arange(rows), np.arange(4 * C), indexing="ij")
    return tiled[((r // 128 * C + b // 4) * 32 + r % 32) * 16 + r % 128 // 32 * 4 + b % 4]


def values(codes, byte, fmt):
    """f64 values [rows, K] of codes [rows, K/2] and scale bytes [rows, blocks] (without g)."""
    nib = np.empty((codes.shape[0], 2 * codes.shape[1]), np.uint8)
    nib[:, 0::2], nib[:, 1::2] = codes & 15, codes >> 4
    v = np.where(nib >= 8, -1.0, 1.0) * GRID[nib & 7]
    s = np.where(byte == 255, np.nan, np.ldexp(1.0, byte.astype(np.int64) - 127)) if fmt == "mx" else E4M3[byte]
    return v * np.repeat(s, BLOCK[fmt], 1)
