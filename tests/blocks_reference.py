"""Microscaled 4-bit blocks written out in 64 bits (test infrastructure)."""
from __future__ import annotations

import numpy as np

VALUES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def blocks_of(d: int) -> int:
    return (d + 127) // 128 * 4


def quantize(x: np.ndarray):
    """Codes [rows, 32 n] (0 .. 15) and scale bytes [rows, n] of x [rows, d]:
    the nearest value by distance, of two at the same distance the one with the
    even code."""
    rows, d = x.shape
    n = blocks_of(d)
    p = np.zeros((rows, 32 * n))
    p[:, :d] = x
    p = p.reshape(rows, n, 32)
    bad = ~np.isfinite(p).all(-1)
    top = np.where(bad, 0.0, np.abs(np.where(np.isfinite(p), p, 0.0)).max(-1))
    mant, e = np.frexp(top)                        # top = mant 2^e, mant in [1/2, 1)
    e = np.where(top > 0, e - 1 - 2, -127).clip(-127, 127)
    y = np.abs(np.where(bad[..., None], 0.0, np.where(np.isfinite(p), p, 0.0))) / np.ldexp(1.0, e)[..., None]
    dist = np.abs(y[..., None] - VALUES)
    rank = dist.min(-1, keepdims=True) == dist
    even = np.arange(8) % 2 == 0
    code = np.where((rank & even).any(-1), (rank & even).argmax(-1), rank.argmax(-1))
    code = code + 8 * (np.signbit(p) & ~bad[..., None])
    return code.reshape(rows, 32 * n).astype(np.uint8), np.where(bad, 255, e + 127).astype(np.uint8)


def pack(codes: np.ndarray) -> np.ndarray:
    return (codes[..., ::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def unpack(codes: np.ndarray) -> np.ndarray:
    return np.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[:-1] + (-1,))


def values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """The numbers of codes [rows, 32 n] (0 .. 15) with scale bytes [rows, n]."""
    v = np.where(codes > 7, -1.0, 1.0) * VALUES[codes & 7]
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(int) - 127))
    return v * np.repeat(s, 32, axis=-1)
