"""Dropout from a counter-based generator (numpy): Philox4x32 with 10 rounds, after
Salmon, Moraes, Dror, Shaw, "Parallel random numbers: as easy as 1, 2, 3" (2011)."""

from __future__ import annotations

import numpy as np

M32 = 0xFFFFFFFF


def philox(counter, key):
    """Four 32-bit words from a counter of four and a key of two, in Python's whole numbers."""
    c, k = list(counter), list(key)
    for _ in range(10):
        p0, p1 = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(p1 >> 32) ^ c[1] ^ k[0], p1 & M32, (p0 >> 32) ^ c[3] ^ k[1], p0 & M32]
        k = [(k[0] + 0x9E3779B9) & M32, (k[1] + 0xBB67AE85) & M32]
    return c


def words(first, n, seed, step=0, site=0):
    """The words of elements first .. first + n - 1 as uint32."""
    at = np.arange(first // 4, (first + n + 3) // 4, dtype=np.uint64)
    c = [at & np.uint64(M32), at >> np.uint64(32), np.full_like(at, step & M32), np.full_like(at, site)]
    k = [seed & M32, seed >> 32 & M32]
    for _ in range(10):
        p0, p1 = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        lo, hi = np.uint64(M32), np.uint64(32)
        c = [(p1 >> hi) ^ c[1] ^ np.uint64(k[0]), p1 & lo, (p0 >> hi) ^ c[3] ^ np.uint64(k[1]), p0 & lo]
        k = [(k[0] + 0x9E3779B9) & M32, (k[1] + 0xBB67AE85) & M32]
    w = np.stack(c, 1).reshape(-1).astype(np.uint32)
    off = first % 4
    return w[off:off + n]


def keep(shape, p, seed, step=0, site=0):
    """Which elements of a dense array of that shape are kept."""
    n = int(np.prod(shape))
    return (words(0, n, seed, step, site).astype(np.int64) >= round(float(np.float32(p)) * 2 ** 32)).reshape(shape)


def forward(x, residual, p, seed, step=0, site=0):
    p = float(np.float32(p))
    k = keep(x.shape, p, seed, step, site)
    y = np.where(k, x / (1 - p), 0.0) if p < 1 else np.zeros_like(x)
    return y if residual is None else residual + y
