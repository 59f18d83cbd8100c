"""fp64 oracle of the 4-bit KV cache: what a row of channels reads back as.

By the definition, a group of 32 channels at a time (the last one of a head may be shorter):
mn = min(0, min x), mx = max(0, max x); s = bf16((mx - mn) * (1 / 15)) with the difference,
the constant and the product in fp32; z = nearest(-mn / s); c = nearest(x / s) + z; z and c held in 0 .. 15; the
group reads back as s * (c - z).  A group without a finite grid reads back as NaN.  The
quotients are taken in fp64, where the quotient of a 24-bit by an 8-bit number cannot round
onto a half that it is not.
"""
from __future__ import annotations

import numpy as np

GROUP = 32
FIFTEENTH = np.float32(1) / np.float32(15)


def bf16(x):
    """Nearest bf16 of fp32 values, ties to even, as fp32."""
    bits = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    bits = (bits + 0x7FFF + ((bits >> 16) & 1)) & 0xFFFF0000
    return bits.astype(np.uint32).view(np.float32)


def readback(x) -> np.ndarray:
    """x [..., head_dim] (values of bf16 or fp32) -> what the cache holds for it, as fp64."""
    x = np.asarray(x, dtype=np.float32)
    out = np.empty(x.shape, dtype=np.float64)
    for lo in range(0, x.shape[-1], GROUP):
        g = x[..., lo:lo + GROUP]
        with np.errstate(over="ignore", invalid="ignore"):
            mn = np.minimum(g.min(-1), np.float32(0))
            mx = np.maximum(g.max(-1), np.float32(0))
            span = (mx - mn).astype(np.float32)
            grid = np.isfinite(span) & np.isfinite(g).all(-1)
            s = bf16(np.where(grid, span, 0).astype(np.float32) * FIFTEENTH).astype(np.float64)
            div = np.where(s > 0, s, 1.0)[..., None]
            flat = (s <= 0)[..., None]
            z = np.clip(np.rint(-np.where(grid, mn, 0).astype(np.float64)[..., None] / div), 0, 15)
            c = np.clip(np.rint(np.where(grid[..., None], g, 0).astype(np.float64) / div) + z, 0, 15)
            val = np.where(flat, 0.0, s[..., None] * (c - z))
        out[..., lo:lo + GROUP] = np.where(grid[..., None], val, np.nan)
    return out
