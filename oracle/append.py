"""Norm and rotation of head rows, and the append to a paged bf16 cache, in fp64.

A token's position on an axis is pos + base; frequency f of a row's first R columns
turns the pair (f, R/2 + f), or (2f, 2f + 1), by position * inv_freq[f].
"""

from __future__ import annotations

import numpy as np

from .attention import bf16_to_f64


def rotate(x, positions, inv_freq, axis, weight=None, eps=0.0, interleaved=False, scale=1.0):
    """fp64 rows [T][H][D] (bf16 bits in), positions [axes][T] whole numbers,
    inv_freq [R/2], axis [R/2]."""
    y = bf16_to_f64(x)
    if weight is not None:
        y = y / np.sqrt((y ** 2).mean(-1, keepdims=True) + eps) * bf16_to_f64(weight)
    out = y.copy()
    half = len(inv_freq)
    for f in range(half):
        # positions beyond fp64's 53 bits do not occur: 31 + 24 bits round once
        angle = positions[axis[f]].astype(np.float64) * float(inv_freq[f])
        i, j = (2 * f, 2 * f + 1) if interleaved else (f, half + f)
        c, s = scale * np.cos(angle)[:, None], scale * np.sin(angle)[:, None]
        out[..., i] = y[..., i] * c - y[..., j] * s
        out[..., j] = y[..., j] * c + y[..., i] * s
    return out
