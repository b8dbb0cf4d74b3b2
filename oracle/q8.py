"""8-bit products with a scale per row (oracle): integers exactly, the rest fp64.

q = rint(v * 127 / amax) of the exact quotient, half to even; scale =
f32(amax / 127).  A row of zeros has scale 0, a row that is not finite has
scale NaN, both q = 0.
"""
from __future__ import annotations

from fractions import Fraction

import numpy as np


def quantise(v, exact: bool = False):
    """(q int8 [R, C], scale f32 [R]) of f32 values; exact=True takes every
    quotient as a fraction of whole numbers (slow), else in fp64, whose error
    (2^-46 at most) no quotient of f32 values comes so near a half."""
    v = np.asarray(v, dtype=np.float32)
    q = np.zeros(v.shape, np.int8)
    scale = np.zeros(v.shape[0], np.float32)
    for r, row in enumerate(v):
        if not np.isfinite(row).all():
            scale[r] = np.nan
            continue
        amax = np.max(np.abs(row))
        scale[r] = np.float32(amax) / np.float32(127)
        if amax == 0:
            continue
        if exact:
            q[r] = [round(Fraction(float(x)) * 127 / Fraction(float(amax))) for x in row]
        else:
            q[r] = np.rint(row.astype(np.float64) * 127.0 / float(amax))
    return q, scale


def matmul(xq, xs, wq, ws):
    """y f64 [T, N] and the exact integer sums int64 [T, N]."""
    acc = np.asarray(xq, np.int64) @ np.asarray(wq, np.int64).T
    return acc * np.asarray(xs, np.float64)[:, None] * np.asarray(ws, np.float64), acc


def swiglu(gu):
    """silu(gate) * up of rows [gate | up], fp64."""
    gu = np.asarray(gu, dtype=np.float64)
    g, u = np.split(gu, 2, axis=-1)
    return g / (1.0 + np.exp(-g)) * u
