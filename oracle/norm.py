"""The norms around a block with its gates and the residual scale (oracle, fp64)."""
from __future__ import annotations

import numpy as np


def sigmoid(v):
    return 1.0 / (1.0 + np.exp(-np.asarray(v, dtype=np.float64)))


def rms_norm(v, w=None, eps: float = 1e-6, offset: float = 0.0):
    """v / sqrt(mean(v^2) + eps) * (w + offset) row by row (w None: a weight of 1)."""
    v = np.asarray(v, dtype=np.float64)
    r = v / np.sqrt(np.mean(v * v, axis=-1, keepdims=True) + eps)
    return r if w is None else r * (np.asarray(w, dtype=np.float64) + offset)


def join(x, y, y2=None, y2_gate=None, w_post=None, gate=None, eps: float = 1e-6, offset: float = 0.0,
         alpha: float = 1.0, beta: float = 1.0):
    """The unrounded new residual stream [T, H].  gate: already activated and
    of a shape that broadcasts to [T, H]."""
    b = np.asarray(y, dtype=np.float64)
    if y2 is not None:
        g = 1.0 if y2_gate is None else sigmoid(y2_gate)[:, None]
        b = b + g * np.asarray(y2, dtype=np.float64)
    if w_post is not None:
        b = rms_norm(b, w_post, eps, offset)
    if gate is not None:
        b = b * gate
    return alpha * np.asarray(x, dtype=np.float64) + beta * b
