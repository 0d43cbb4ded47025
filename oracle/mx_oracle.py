"""Float64 oracle of microscaled 4-bit matrices: the definition, value by value.

A block of 32 values shares 2^e, e = max(floor(log2 max|x|) - 2, -127); each value is the nearest of +-{0, 1/2, 1,
3/2, 2, 3, 4, 6} times 2^e, ties to the even place in that list, larger ones 6.  Codes two a byte, the first in the
low half, the sign in the code's highest bit; scale byte e + 127, 255 for a block with a NaN or an infinity.  Rows are
padded to a multiple of 256 values with zero codes; blocks past the end have scale byte 0."""

from __future__ import annotations

import math

import numpy as np

LEVELS = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def padded(cols: int) -> int:
    return -(-cols // 256) * 256


def nearest(y: float) -> int:
    """Place of the level nearest to y >= 0: the smaller distance, then the even place."""
    return min(range(8), key=lambda i: (abs(min(y, 6.0) - LEVELS[i]), i % 2))


def quantize_block(x) -> tuple[list[int], int]:
    x = [float(v) for v in x]
    if any(not math.isfinite(v) for v in x):
        return [0] * len(x), 255
    m = max(abs(v) for v in x)
    e = -127 if m == 0 else max(math.frexp(m)[1] - 1 - 2, -127)
    return [nearest(abs(v) / math.ldexp(1.0, e)) | (8 if math.copysign(1.0, v) < 0 else 0) for v in x], e + 127


def quantize(x: np.ndarray) -> tuple[np.ndarray, np.ndarray]:
    rows, cols = x.shape
    full = np.zeros((rows, padded(cols)))
    full[:, :cols] = x
    codes = np.zeros((rows, full.shape[1] // 2), dtype=np.uint8)
    scales = np.zeros((rows, full.shape[1] // 32), dtype=np.uint8)
    for r in range(rows):
        for b in range(scales.shape[1]):
            c, s = quantize_block(full[r, 32 * b:32 * b + 32])
            scales[r, b] = s
            codes[r, 16 * b:16 * b + 16] = [c[2 * i] | c[2 * i + 1] << 4 for i in range(16)]
    return codes, scales


def values(codes: np.ndarray, scales: np.ndarray, cols: int) -> np.ndarray:
    """What an MX matrix holds, float64 [rows, cols]."""
    nib = np.stack([codes & 15, codes >> 4], axis=-1).reshape(codes.shape[0], -1)
    v = np.array(LEVELS)[nib & 7] * np.where(nib & 8, -1.0, 1.0)
    e = np.repeat(scales.astype(np.int64) - 127, 32, axis=1)
    v = np.ldexp(v, e)
    v[np.repeat(scales == 255, 32, axis=1)] = np.nan
    return v[:, :cols]


def silu(g):
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g))


def product(a: np.ndarray, w: np.ndarray, act: str = "none"):
    """(y, mag): a w^T (gated for "swiglu": w holds the gate rows, then the up rows) and, per plain sum, the sum of
    the terms' magnitudes, which bounds its rounding."""
    y, mag = a @ w.T, np.abs(a) @ np.abs(w).T
    return (y, mag) if act == "none" else (silu(y[:, :w.shape[0] // 2]) * y[:, w.shape[0] // 2:], mag)
