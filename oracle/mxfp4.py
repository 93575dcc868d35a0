"""MXFP4 rows and products in fp64 (test infrastructure, numpy).

quantize: OCP Microscaling v1.0 conversion with the E2M1 element, written from
the definition: the nearest representable magnitude, a tie to the even code.
matmul: the products' definition on the values that codes and scales stand
for, and the magnitude sum that its error bounds use.
"""
from __future__ import annotations

import numpy as np

MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quantize(x: np.ndarray):
    """codes uint8 [R, K/2] and scales uint8 [R, K/32] of rows x [R, K] (values exact in fp64)"""
    x = np.asarray(x, dtype=np.float64)
    R, K = x.shape
    b = x.reshape(R, K // 32, 32)
    amax = np.abs(b).max(axis=2)
    bad = ~np.isfinite(amax)
    _, e = np.frexp(np.where(bad, 1.0, amax))          # amax = m 2^e, m in [0.5, 1)
    e = np.where(amax == 0, -127, np.maximum(e - 1 - 2, -127))
    scales = np.where(bad, 255, e + 127).astype(np.uint8)
    v = np.abs(np.where(bad[..., None], 0.0, b)) / np.exp2(e.astype(np.float64))[..., None]
    codes = np.zeros(v.shape, dtype=np.uint8)
    for i in range(7):
        mid = (MAGNITUDES[i] + MAGNITUDES[i + 1]) / 2
        codes += (v >= mid) if i % 2 == 1 else (v > mid)  # the tie at a midpoint below an even code goes up
    codes |= np.where(np.signbit(b), 8, 0).astype(np.uint8)
    codes = np.where(bad[..., None], 7, codes).reshape(R, K).astype(np.uint8)
    return codes[:, 0::2] | (codes[:, 1::2] << 4), scales


def values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """fp64 [.., K] of codes [.., K/2] and row-major scales [.., K/32]"""
    c = np.stack([codes & 15, codes >> 4], axis=-1).reshape(*codes.shape[:-1], -1)
    m = np.where(c >= 8, -1.0, 1.0) * MAGNITUDES[c & 7]
    s = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127))
    return m * np.repeat(s, 32, axis=-1)


def tile_scales(scales: np.ndarray, swiglu: bool = False) -> np.ndarray:
    """[E, ceil(N/128), ceil(K/128), 512] of scales [E, N, K/32], byte by byte"""
    E, N, nb = scales.shape
    out = np.zeros((E, -(-N // 128), -(-nb // 4), 512), dtype=np.uint8)
    for row in range(N):
        src = (row % 2) * (N // 2) + row // 2 if swiglu else row
        at = 16 * (row % 32) + 4 * (row % 128 // 32)
        for b in range(nb):
            out[:, row // 128, b // 4, at + b % 4] = scales[:, src, b]
    return out


def tiled_scale(tiled: np.ndarray, row: int, b: int):
    """the byte of (row, b) in tiles [row tiles, ceil(K/128), 512]"""
    return tiled[row // 128, b // 4, 16 * (row % 32) + 4 * (row % 128 // 32) + b % 4]


def matmul(a: np.ndarray, w: np.ndarray):
    """a [M, K], w [N, K] (fp64 values): y = a w^T and |a| |w|^T"""
    return a @ w.T, np.abs(a) @ np.abs(w).T


def swiglu(y: np.ndarray) -> np.ndarray:
    g, u = np.split(y, 2, axis=-1)
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g)) * u
