"""MXFP4 and token sorting in numpy, fp64, from the definitions.

MXFP4 (OCP microscaling formats, E2M1 elements with an E8M0 scale per 32
values): scale exponent floor(log2 max|x|) - 2, clamped to the range of a
biased byte; elements to the nearest representable value, ties to even.
"""
from __future__ import annotations

import numpy as np

VALUES = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=np.float64)


def quantize(x: np.ndarray):
    """x [rows, cols] -> (codes [rows, cols] 0..15, scale bytes [rows, cols / 32])."""
    rows, cols = x.shape
    v = np.asarray(x, dtype=np.float64).reshape(rows, cols // 32, 32)
    s = np.zeros(v.shape[:2], dtype=np.int64)
    codes = np.zeros(v.shape, dtype=np.uint8)
    for r in range(rows):
        for b in range(cols // 32):
            blk = v[r, b]
            if not np.all(np.isfinite(blk)):
                s[r, b] = 255
                continue
            top = np.max(np.abs(blk))
            s[r, b] = max(np.frexp(top)[1] - 1 - 2 + 127, 0) if top > 0 else 0
            q = np.ldexp(np.abs(blk), 127 - int(s[r, b]))
            d = np.abs(q[:, None] - VALUES[None, :])
            near = d == d.min(axis=1, keepdims=True)
            # a tie is between neighbours, one of which has an even code
            even = np.argmax(near & (np.arange(8) % 2 == 0), axis=1)
            first = np.argmax(near, axis=1)
            code = np.where(near.sum(1) > 1, even, first)
            codes[r, b] = code + 8 * np.signbit(blk)
    return codes.reshape(rows, cols), s.astype(np.uint8)


def values(codes: np.ndarray, s: np.ndarray) -> np.ndarray:
    mag = VALUES[codes & 7]
    v = np.where(codes & 8, -mag, mag).reshape(*s.shape, 32)
    out = np.ldexp(v, s.astype(np.int64)[..., None] - 127)
    return np.where((s == 255)[..., None], np.nan, out).reshape(codes.shape)


def pack(codes: np.ndarray) -> np.ndarray:
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)


def unpack(packed: np.ndarray) -> np.ndarray:
    out = np.empty((packed.shape[0], packed.shape[1] * 2), dtype=np.uint8)
    out[:, 0::2], out[:, 1::2] = packed & 15, packed >> 4
    return out


def tile(s: np.ndarray) -> np.ndarray:
    """Scale bytes [rows, blocks] to [ceil(rows / 128), ceil(blocks / 4), 512], zeros outside."""
    rows, blocks = s.shape
    out = np.zeros((-(-rows // 128), -(-blocks // 4), 512), dtype=np.uint8)
    for r in range(rows):
        for b in range(blocks):
            out[r // 128, b // 4, (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4] = s[r, b]
    return out


def untile(t: np.ndarray, rows: int, cols: int) -> np.ndarray:
    r, b = np.arange(rows)[:, None], np.arange(cols // 32)[None, :]
    return t[r // 128, b // 4, (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4]


def decode(packed: np.ndarray, tiles: np.ndarray) -> np.ndarray:
    rows, cols = packed.shape[0], packed.shape[1] * 2
    return values(unpack(packed), untile(tiles, rows, cols))


def round_trip(x: np.ndarray) -> np.ndarray:
    return values(*quantize(x))


def sort(ids: np.ndarray, n_experts: int):
    """(order, position, offsets) of the pairs by expert, dropped pairs -1."""
    flat = ids.reshape(-1)
    kept = sorted((int(e), i) for i, e in enumerate(flat) if 0 <= e < n_experts)
    order = np.full(flat.size, -1, dtype=np.int32)
    position = np.full(flat.size, -1, dtype=np.int32)
    for p, (_, i) in enumerate(kept):
        order[p], position[i] = i, p
    offsets = np.array([sum(e < n for e, _ in kept) for n in range(n_experts + 1)], dtype=np.int32)
    return order, position.reshape(ids.shape), offsets


def silu(z: np.ndarray) -> np.ndarray:
    return z / (1 + np.exp(-z))
