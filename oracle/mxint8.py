"""MXINT8 (OCP microscaling, 8-bit integer elements), SwiGLU and its gradients, in
fp64 on the CPU.

A block of 32 values shares X = 2^(s - 127), s the fp32 exponent field of the
largest magnitude (0 for subnormal numbers and zero); a code is the nearest integer
to 64 x / X, even at ties, within +-127. An infinity or a NaN makes the block NaN
(s = 255, codes 0).
"""
from __future__ import annotations

import numpy as np


def scale_of(top: float) -> int:
    """s from the largest magnitude of a block."""
    if not np.isfinite(top):
        return 255
    if top < 2.0 ** -126:
        return 0
    return int(np.floor(np.log2(top))) + 127 if top == 2.0 ** np.floor(np.log2(top)) else int(np.frexp(top)[1]) - 1 + 127


def quantize(x: np.ndarray):
    """Rows x [rows, cols] -> (codes int8 [rows, cols], scales uint8 [rows, ceil(cols / 32)])."""
    x = np.asarray(x, dtype=np.float64)
    rows, cols = x.shape
    codes = np.zeros((rows, cols), np.int8)
    scales = np.zeros((rows, -(-cols // 32)), np.uint8)
    for r in range(rows):
        for b in range(scales.shape[1]):
            v = x[r, 32 * b:32 * b + 32]
            s = scale_of(float(np.max(np.abs(v)))) if np.all(np.isfinite(v)) else 255
            scales[r, b] = s
            if s != 255:
                codes[r, 32 * b:32 * b + 32] = np.clip(np.rint(v * 64 * 2.0 ** (127 - s)), -127, 127)
    return codes, scales


def dequantize(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    s = np.repeat(scales.astype(np.int64), 32, axis=1)[:, :codes.shape[1]]
    return np.where(s == 255, np.nan, codes.astype(np.float64) * 2.0 ** (np.minimum(s, 254) - 133.0))


def logistic(g):
    with np.errstate(over="ignore"):
        return 1 / (1 + np.exp(-np.asarray(g, np.float64)))


def swiglu(g, u):
    return g * logistic(g) * u


def swiglu_backward(g, u, gh, c):
    """(gg, gu, c h, gradient of c) of rows of h = silu(g) u that enter a sum as c h."""
    s, c = logistic(g), np.asarray(c, np.float64)[:, None]
    h = g * s * u
    return c * gh * u * s * (1 + g * (1 - s)), c * gh * g * s, c * h, (gh * h).sum(1)
