"""Scored top-k routing (oracle, fp64): softmax or sigmoid scores, a bias that
counts for the selection only, groups of experts, top-k, renormalised and
scaled weights.  Written with plain loops over one token at a time.

Scores and their sums are fp64; without a bias an expert's logit stands for
its score wherever scores are only compared.  Every tie goes to the lower
index.  An expert with a logit or bias of -inf or NaN is masked: score 0, no
member of its group's sum, behind every live expert.
"""
from __future__ import annotations

import math

import numpy as np

F32_MAX = float(np.finfo(np.float32).max)


def _scores(l, live, sigmoid: bool):
    s = np.zeros(len(l))
    if sigmoid:
        for e in np.flatnonzero(live):
            x = float(l[e])
            s[e] = 1.0 / (1.0 + math.exp(-x)) if x > -700.0 else math.exp(max(x, -740.0))
    elif live.any():
        z = np.exp(l[live] - l[live].max())
        s[live] = z / z.sum()
    return s


def route_row(logits, k: int, sigmoid: bool = False, bias=None, n_groups: int = 1, topk_groups: int = 1,
              group_top: int = 1, renormalise: bool = True, scale: float = 1.0):
    """(idx, weights) of one token; logits [E] as read (f32 values)."""
    l = np.minimum(np.asarray(logits, dtype=np.float64), F32_MAX)
    E = len(l)
    b = np.zeros(E) if bias is None else np.asarray(bias, dtype=np.float64)
    live = (l > -np.inf) & (b > -np.inf)                # False for NaN too
    s = _scores(l, live, sigmoid)
    by = l if bias is None else s + b                   # what experts are compared by
    size = E // n_groups
    standing = []
    for g in range(n_groups):
        members = [e for e in range(g * size, (g + 1) * size) if live[e]]
        if group_top == 1:
            top = max((by[e] for e in members), default=-np.inf)
        else:
            top = sum(sorted((s[e] + b[e] for e in members), reverse=True)[:2]) if members else -np.inf
        standing.append((-top, g))
    kept = {g for _, g in sorted(standing)[:topk_groups]}
    order = sorted((e for e in range(E) if e // size in kept),
                   key=lambda e: (0, -by[e], e) if live[e] else (1, 0.0, e))
    idx = np.array(order[:k], dtype=np.int32)
    if not renormalise:
        return idx, s[idx] * scale
    # ratios of scores that underflow together: relative to the largest selected
    w = np.zeros(k)
    on = live[idx]
    if on.any():
        li = l[idx][on]
        e = np.minimum(li, 0.0) if sigmoid else li
        v = np.exp(e - e.max())
        if sigmoid:
            v = v / (1.0 + np.exp(-np.abs(li)))
        w[on] = v / v.sum()
    return idx, w * scale


def route(logits, k: int, **rule):
    """(idx int32 [T, k], weights f64 [T, k])."""
    rows = [route_row(r, k, **rule) for r in np.asarray(logits)]
    return np.stack([i for i, _ in rows]), np.stack([w for _, w in rows])
