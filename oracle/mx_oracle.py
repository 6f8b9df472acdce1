"""fp64 definitions of the block-scaled formats and the product of two matrices
held in them (numpy, written from the formats' definition; test use only).

A block is 32 consecutive elements of a row, its scale the smallest power of two
s >= 2^-127 with max |x| <= top * s; its elements are the grid points nearest
x / s, ties to the even code."""

from __future__ import annotations

import numpy as np

BLOCK = 32
GRIDS = {"mx4": np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6]), "mx8": np.arange(128, dtype=np.float64)}


def quantise(x, fmt):
    """codes (magnitude index), negative (bool) and scale bytes of x [rows][cols]."""
    x = np.asarray(x, dtype=np.float64)
    rows, cols = x.shape
    grid = GRIDS[fmt]
    b = x.reshape(rows, cols // BLOCK, BLOCK)
    finite = np.isfinite(b).all(-1)
    most = np.where(finite, np.abs(np.where(np.isfinite(b), b, 0)).max(-1), 0)
    e = np.full(most.shape, -127)
    for k in range(-127, 128):  # raise the exponent until the block fits
        e = np.where(most > grid[-1] * 2.0 ** e.astype(np.float64), k, e)
    s = 2.0 ** e.astype(np.float64)
    v = np.abs(np.where(finite[..., None], b, 0)) / s[..., None]
    up = np.searchsorted(grid, v, side="left")          # first grid point >= v
    up = np.minimum(up, len(grid) - 1)
    lo = np.maximum(up - 1, 0)
    d_lo, d_up = v - grid[lo], grid[up] - v
    pick = np.where((d_up < d_lo) | ((d_up == d_lo) & (up % 2 == 0)), up, lo)
    # a value of 2^128 has no fp32: the element below
    pick = np.where(grid[pick] * s[..., None] >= 2.0 ** 128, pick - 1, pick)
    neg = np.signbit(b) & finite[..., None]
    byte = np.where(finite, e + 127, 255).astype(np.uint8)
    return pick.reshape(rows, cols), neg.reshape(rows, cols), byte


def values(x, fmt):
    """What x stands for once packed."""
    mag, neg, byte = quantise(x, fmt)
    return _values(mag, neg, byte, fmt)


def _values(mag, neg, byte, fmt):
    s = np.where(byte == 255, np.nan, 2.0 ** (byte.astype(np.float64) - 127))
    v = GRIDS[fmt][mag] * np.repeat(s, BLOCK, axis=1)
    return np.where(neg, -v, v)


def pack(x, fmt):
    """(q, byte [rows][cols/32]) as stored."""
    mag, neg, byte = quantise(x, fmt)
    rows, cols = mag.shape
    if fmt == "mx4":
        n = (mag | (neg << 3)).astype(np.uint8)
        return n[:, 0::2] | (n[:, 1::2] << 4), byte
    c = (mag | (neg << 7)).astype(np.uint8)
    out = np.empty_like(c)
    for i, e in enumerate((0, 2, 1, 3)):  # byte i of a group of four holds element e
        out[:, i::4] = c[:, e::4]
    return out, byte


def tile_scales(byte):
    """Scale bytes [rows][blocks] in the stored order (0 outside)."""
    rows, blocks = byte.shape
    kt = -(-blocks // 4)
    out = np.zeros(-(-rows // 128) * kt * 512, np.uint8)
    r, b = np.meshgrid(np.arange(rows), np.arange(blocks), indexing="ij")
    out[((r // 128) * kt + b // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4] = byte
    return out


def untile_scales(tiles, rows, cols):
    r, b = np.meshgrid(np.arange(rows), np.arange(cols // BLOCK), indexing="ij")
    kt = -(-cols // 128)
    return tiles[((r // 128) * kt + b // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4]


def unpack(q, byte, fmt):
    """Values of stored bytes, element by element."""
    rows = q.shape[0]
    if fmt == "mx4":
        n = np.empty((rows, 2 * q.shape[1]), np.uint8)
        n[:, 0::2], n[:, 1::2] = q & 15, q >> 4
        return _values(n & 7, (n & 8) != 0, byte, fmt)
    c = np.empty_like(q)
    for i, e in enumerate((0, 2, 1, 3)):
        c[:, e::4] = q[:, i::4]
    return _values(c & 127, (c & 128) != 0, byte, fmt)


def gemm(xv, wv):
    """Y = X W^T and the sums of the terms' magnitudes."""
    return xv @ wv.T, np.abs(xv) @ np.abs(wv).T
