"""Appending with rotation and rows in 4 bits, in 64 bits from the definitions in the
header, on numpy arrays. Shares no code with the library."""
from __future__ import annotations

import numpy as np

MOST = 30656.0


def rotate(x, pos, theta: float, half: bool = False, band_axis=None):
    """Row x [d] at positions pos [axes]: band f times e^{i w_f p}."""
    d = x.shape[-1]
    x = x.astype(np.float64)
    out = np.empty_like(x)
    for f in range(d // 2):
        p = float(pos[0 if band_axis is None else band_axis[f]])
        a, b = (f, f + d // 2) if half else (2 * f, 2 * f + 1)
        c, s = np.cos(p * theta ** (-2.0 * f / d)), np.sin(p * theta ** (-2.0 * f / d))
        out[..., a] = x[..., a] * c - x[..., b] * s
        out[..., b] = x[..., a] * s + x[..., b] * c
    return out


def nibble(d: int, e: int) -> int:
    """Number of the nibble that holds element e's code."""
    j, i = divmod(e, d // 4)
    return 8 * (4 * (i // 8) + j) + i % 8 if d == 128 else 8 * (2 * (i // 4) + j // 2) + 4 * (i % 4 // 2) + 2 * (j % 2) + i % 2


def quantise(x):
    """Row x [d] (fp64): (codes [d], scale [4], minimum [4]), the pairs fp16 values; a NaN makes its quarter NaN."""
    d = x.shape[-1]
    codes, scale, low = np.zeros(d, dtype=np.int64), np.zeros(4), np.zeros(4)
    for j in range(4):
        g = x[j * d // 4:(j + 1) * d // 4].astype(np.float64)
        if np.isnan(g).any():
            scale[j] = low[j] = np.nan
            continue
        g = np.clip(g, -MOST, MOST)
        low[j] = np.float64(np.float16(g.min()))
        scale[j] = np.float64(np.float16(max(0.0, g.max() - low[j]) / 15))
        if scale[j] > 0:
            codes[j * d // 4:(j + 1) * d // 4] = np.clip(np.rint((g - low[j]) / scale[j]), 0, 15)
    return codes, scale, low


def pack(x):
    """Row x [d] as bytes [d / 2 + 16]."""
    d = x.shape[-1]
    codes, scale, low = quantise(x)
    out = np.zeros(d // 2 + 16, dtype=np.uint8)
    for e in range(d):
        n = nibble(d, e)
        out[n // 2] |= codes[e] << (4 * (n % 2))
    out[d // 2:] = np.stack([scale, low], 1).astype(np.float16).reshape(-1).view(np.uint8)
    return out


def values(rows):
    """Bytes [..., d / 2 + 16] to the fp64 values [..., d] they stand for."""
    rows = np.asarray(rows)
    d = (rows.shape[-1] - 16) * 2
    pairs = np.ascontiguousarray(rows[..., d // 2:]).view(np.float16).astype(np.float64)
    n = np.array([nibble(d, e) for e in range(d)])
    codes = (rows[..., n // 2] >> (4 * (n % 2)).astype(np.uint8)) & 15
    j = np.arange(d) // (d // 4)
    return pairs[..., 2 * j + 1] + pairs[..., 2 * j] * codes
