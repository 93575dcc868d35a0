"""Rows in 8-bit floating point (E4M3, a power-of-two scale for 128 elements) in
fp64 (test infrastructure, numpy), written from the definition: all 256 codes in
a table, the nearest value, a tie to the even code.
"""
from __future__ import annotations

import numpy as np


def _value(code: int) -> float:
    sign, e, m = -1.0 if code & 128 else 1.0, (code >> 3) & 15, code & 7
    if e == 15 and m == 7:
        return float("nan")
    return sign * (m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))


VALUES = np.array([_value(c) for c in range(256)])
MAGNITUDES = VALUES[:127]                       # codes 0 .. 126, ascending; 126 is 448


def quantize(x: np.ndarray):
    """codes uint8 [R, K] and scales uint8 [R, ceil(K/128)] of rows x [R, K] (values exact in fp64)"""
    x = np.asarray(x, dtype=np.float64)
    R, K = x.shape
    codes = np.zeros((R, K), dtype=np.uint8)
    scales = np.zeros((R, -(-K // 128)), dtype=np.uint8)
    mids = (MAGNITUDES[:-1] + MAGNITUDES[1:]) / 2
    for r in range(R):
        for b in range(scales.shape[1]):
            v = x[r, 128 * b:128 * b + 128]
            at = slice(128 * b, 128 * b + v.size)
            if not np.isfinite(v).all():
                codes[r, at], scales[r, b] = 127, 255
                continue
            amax, e = np.abs(v).max(), -127
            while amax > 448 * 2.0 ** e:
                e += 1
            scales[r, b] = e + 127
            m = np.abs(v) / 2.0 ** e
            c = np.searchsorted(mids, m, side="left")      # midpoints below m
            tie = (c < 126) & (mids[np.minimum(c, 125)] == m) & (c % 2 == 1)
            codes[r, at] = np.minimum(c + tie, 126) | np.where(np.signbit(v), 128, 0)
    return codes, scales


def row_values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """fp64 [R, K] of codes [R, K] with a scale for 128 elements"""
    s = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127))
    return VALUES[codes] * np.repeat(s, 128, axis=1)[:, :codes.shape[1]]


def weight_values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """fp64 [N, K] of codes [N, K] with a scale for 128 x 128"""
    return row_values(codes, np.repeat(scales, 128, axis=0)[:codes.shape[0]])


def tile_scales(scales: np.ndarray, N: int, swiglu: bool = False) -> np.ndarray:
    """[E, ceil(N/128), ceil(K/128), 512] of scales [E, ceil(N/128), ceil(K/128)], byte by byte"""
    E, rt, kt = scales.shape
    out = np.zeros((E, rt, kt, 512), dtype=np.uint8)
    for row in range(N):
        src = (row % 2) * (N // 2) + row // 2 if swiglu else row
        at = 16 * (row % 32) + 4 * (row % 128 // 32)
        out[:, row // 128, :, at:at + 4] = scales[:, src // 128, :, None]
    return out
