"""Plain 64-bit forms of 4-bit pools (e2m1 numbers under a power of two per 32
dims): numbers and scales of rows, the values that they stand for, and where a
page holds them.  numpy on the host; knows nothing of the library."""
from __future__ import annotations

import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
NAN_SCALE = 255


def row_bytes(H, D):
    return (H * D * 17 // 32 + 15) // 16 * 16


def quantise(x, scale=1.0):
    """Codes [.., D] (0..15) and scale bytes [.., D / 32] of float32 x [.., D]:
    each block's quotients x / scale, rounded to 32 bits, under the smallest
    2^e (-23 <= e <= 13) with max <= 7 * 2^e, to the nearest of GRID * 2^e (a tie
    to the even code, past 6 to 6).  A block with a NaN is 255 and zeros."""
    x = np.asarray(x, np.float32)
    with np.errstate(all="ignore"):
        y = x if scale == 1.0 else (x / np.float32(scale)).astype(np.float32)
    y = y.astype(np.float64).reshape(*x.shape[:-1], -1, 32)
    nan = np.isnan(y).any(-1)
    a = np.abs(np.where(nan[..., None], 0.0, y))
    top = a.max(-1)
    e = np.full(top.shape, -23)
    for k in range(-22, 14):
        e = np.where(top > 7.0 * 2.0 ** (k - 1), k, e)
    a = np.minimum(a / 2.0 ** e[..., None], 8.0)
    far = np.abs(a[..., None] - GRID)                   # exact: both are short
    best = far.min(-1, keepdims=True)
    even = np.where(far == best, np.arange(8) % 2, 9)   # of two equally near the even one
    code = even.argmin(-1)
    code = np.where(a >= 6.0, 7, code)
    code = code + 8 * np.signbit(y)
    code = np.where(nan[..., None], 0, code)
    return code.reshape(x.shape).astype(np.uint8), np.where(nan, NAN_SCALE, e + 127).astype(np.uint8)


def values(codes, scales):
    """float64 values [.., D] of codes and scale bytes."""
    v = np.where(codes & 8, -1.0, 1.0) * GRID[codes & 7]
    s = 2.0 ** (scales.astype(np.float64) - 127.0)
    s = np.where(scales == NAN_SCALE, np.nan, s)
    return v * np.repeat(s, 32, -1)


def pack(codes):
    return (codes[..., 0::2] | codes[..., 1::2] << 4).astype(np.uint8)


def unpack(b):
    return np.stack([b & 15, b >> 4], -1).reshape(*b.shape[:-1], -1)


def views(plane, page, H, D, layout):
    """Number bytes [pages, page, H, D / 2] and scale bytes [pages, page, H, D / 32]
    of a plane [pages, page * row_bytes] uint8, as views."""
    P = plane.shape[0]
    if layout == "nhd":
        rows = plane.reshape(P, page, -1)
        n = H * D // 2
        return (rows[..., :n].reshape(P, page, H, D // 2, copy=False),
                rows[..., n:n + H * D // 32].reshape(P, page, H, D // 32, copy=False))
    n = H * page * D // 2
    return (plane[:, :n].reshape(P, H, page, D // 2, copy=False).transpose(0, 2, 1, 3),
            plane[:, n:n + H * page * D // 32].reshape(P, H, page, D // 32, copy=False)
            .transpose(0, 2, 1, 3))
