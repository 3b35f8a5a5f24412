"""Oracle of the rotations by position (include/apr_rope.h), in float64 with float32 roundings where the definition has them.

Plain numpy; nothing is shared with the CUDA library. A table is float32 [positions][pairs][2].
"""

from __future__ import annotations

import numpy as np


def _f32(x):
    return np.asarray(x, np.float64).astype(np.float32).astype(np.float64)


def rope_table(inv_freq, first, positions, scale=1.0):
    """float64 [positions][pairs][2]. Position times float32 frequency, up to 54 bits, is exact in a long double (64 bits
    or more)."""
    angle = np.arange(first, first + positions).astype(np.longdouble)[:, None] * np.asarray(inv_freq, np.float32).astype(np.longdouble)
    return (np.stack((np.cos(angle), np.sin(angle)), -1) * np.longdouble(scale)).astype(np.float64)


def rope_rows(table, pair_axis, interleaved, positions, x, heads, norm=None, eps=0.0):
    """Rows x (float32 values [rows][heads * dim]) normed and rotated: float32 values [rows][heads * dim]. positions
    [axes][rows]; pair_axis None: axis 0. (The sum of squares is in float64; each later step is a float64 one of two
    float32 numbers, rounded to float32.)"""
    x = np.asarray(x, np.float32)
    rows, pairs = x.shape[0], table.shape[1]
    y = x.astype(np.float64).reshape(rows, heads, x.shape[1] // heads)
    if norm is not None:
        with np.errstate(divide="ignore", invalid="ignore"):
            r = _f32(1.0 / np.sqrt((y * y).mean(-1, keepdims=True) + np.float64(np.float32(eps))))
            y = _f32(_f32(y * r) * np.asarray(norm, np.float32).astype(np.float64))
    out = y.copy()
    for i in range(pairs):
        axis = 0 if pair_axis is None else int(pair_axis[i])
        turn = np.asarray(table, np.float32)[np.asarray(positions)[axis], i].astype(np.float64)[:, None]
        lo, hi = (2 * i, 2 * i + 1) if interleaved else (i, pairs + i)
        a, b = y[..., lo], y[..., hi]
        out[..., lo] = _f32(_f32(a * turn[..., 0]) - _f32(b * turn[..., 1]))
        out[..., hi] = _f32(_f32(b * turn[..., 0]) + _f32(a * turn[..., 1]))
    return out.astype(np.float32).reshape(x.shape)
