"""The microscaled 4-bit operators in float64 (and exact rational steps), written from the format's definition on numpy."""
import numpy as np

VALUES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def scale_at(rows, K):
    """Offsets [rows, K / 32] of the blocks' scales in the tiles, and their size in bytes."""
    r, b = np.arange(rows)[:, None], np.arange(K // 32)[None]
    across = -(-K // 128)
    at = ((r // 128) * across + b // 4) * 512 + 16 * (r % 32) + 4 * (r % 128 // 32) + b % 4
    return at, -(-rows // 128) * across * 512


def quantize(x):
    """(codes, scale bytes [rows, K / 32]) of x [rows, K]: the nearest value by distance, ties to the even code."""
    x = np.asarray(x, np.float64)
    b = x.reshape(x.shape[0], -1, 32)
    bad = ~np.isfinite(b).all(-1)
    f = np.where(bad[..., None], 0.0, b)
    most = np.abs(f).max(-1)
    _, e = np.frexp(most)                                   # most = m * 2 ** e, 0.5 <= m < 1
    s = np.where(most > 0, np.maximum(e - 1 - 2, -127), -127)
    q = np.abs(f) / np.exp2(s)[..., None]                   # exact: a power of two
    dist = np.abs(q[..., None] - VALUES)
    least = dist.min(-1, keepdims=True)
    near = dist == least                                    # one code, or two neighbours of which one is even
    even = near & (np.arange(8) % 2 == 0)
    code = np.where(even.any(-1), even.argmax(-1), near.argmax(-1))
    code = np.where(np.signbit(f), code + 8, code)
    return code.reshape(x.shape).astype(np.uint8), np.where(bad, 255, s + 127).astype(np.uint8)


def values(codes, scales):
    """float64 values [rows, K] of codes [rows, K] and scale bytes [rows, K / 32]."""
    v = np.where(codes >= 8, -1.0, 1.0) * VALUES[codes & 7]
    s = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127))
    with np.errstate(invalid="ignore"):
        return (v.reshape(v.shape[0], -1, 32) * s[..., None]).reshape(v.shape)


def pack(codes):
    return (codes[..., ::2] | (codes[..., 1::2] << 4)).astype(np.uint8).view(np.int32)


def unpack(packed):
    b = np.ascontiguousarray(packed).view(np.uint8)
    return np.stack((b & 15, b >> 4), -1).reshape(*b.shape[:-1], -1)


def tiles(scales, fill=0):
    """Scale bytes [rows, K / 32] in tiles; `fill` for rows past the last (blocks past K are 0)."""
    rows, blocks = scales.shape
    at, size = scale_at(rows, blocks * 32)
    out = np.zeros(size, np.uint8)
    every, _ = scale_at(-(-rows // 128) * 128, -(-blocks // 4) * 128)
    out[every[rows:]] = fill
    out[at] = scales
    return out


def product(x, w, gated=False):
    """(y, bound of what float32 sums may be off by) of float64 x [M, K] and w [N, K] or [2, N, K].

    A product of two codes and two powers of two is exact.  The tensor core adds 64 of them to a running sum: 64 terms cut to
    the last bit of the largest, 2 ** -23 of it or less each, then one rounding of the sum, K / 64 times."""
    each = (x.shape[1] / 64 + 65) * 2.0 ** -23

    def one(m):
        return x @ m.T, each * (np.abs(x) @ np.abs(m).T)
    with np.errstate(invalid="ignore", over="ignore"):
        if not gated:
            return one(w)
        (g, dg), (u, du) = one(w[0]), one(w[1])
        s = 1 / (1 + np.exp(-g))
        y = g * s * u
        # silu's slope is at most 1.1; exp, the quotient and two products are a few roundings: 2 ** -20 in all
        return y, 1.1 * dg * (np.abs(u) + du) + np.abs(g * s) * du + np.abs(y) * 2.0 ** -20
