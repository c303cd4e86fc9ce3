"""The choice of experts from router logits, restated in float64.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

The pages take ids and weights as inputs; what is fixed here:

* s = softmax(z) or sigmoid(z), c = s + bias, without a bias the order of z;
* a NaN or -inf in a logit takes the expert out altogether, in a bias out of the
  choice and its group's value (the softmax has its logit still);
* groups of neighbouring experts count with the sum of their ``group_top``
  largest c (of what they have; by z where that is one score without a bias);
  the ``top_groups`` best stay;
* the top_k largest c in descending order, ties (of groups too) to the lowest
  index; id -1 and weight 0 where none is left;
* weights are s, over their sum where renormalised, times a constant.
"""

from __future__ import annotations

import numpy as np


def scores(z, score):
    """s of one row of logits, 0 for experts that are out."""
    z = np.asarray(z, dtype=np.float64)
    live = z > -np.inf  # (False for NaN)
    s = np.zeros(z.shape)
    if not live.any():
        return s
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            s[live] = 1.0 / (1.0 + np.exp(-z[live]))
        return s
    top = z[live].max()
    e = np.where(z[live] == top, 1.0, np.exp(np.minimum(z[live], 1e308) - top)) if np.isfinite(top) else (z[live] == top) * 1.0
    s[live] = e / e.sum()
    return s


def route_row(z, bias, top_k, score, renorm=True, scale=1.0, groups=1, top_groups=None, group_top=1):
    """(ids [top_k], weights [top_k]) of one token."""
    z = np.asarray(z, dtype=np.float64)
    n = z.shape[0]
    s = scores(z, score)
    out = ~(z > -np.inf)
    c = s.copy()
    if bias is not None:
        b = np.asarray(bias, dtype=np.float64)
        out |= ~(b > -np.inf)
        c = np.where(out, 0.0, s + np.where(out, 0.0, b))
    if groups > 1:
        per = n // groups
        value = []
        for g in range(groups):
            by = z if bias is None and group_top == 1 else c  # (largest c without a bias: the order of z)
            mine = sorted((by[e] for e in range(g * per, (g + 1) * per) if not out[e]), reverse=True)
            value.append(sum(mine[:group_top]) if mine else -np.inf)
        kept = sorted(range(groups), key=lambda g: (-value[g], g))[: groups if top_groups is None else top_groups]
        for g in range(groups):
            if g not in kept:
                out[g * per:(g + 1) * per] = True
    key = z if bias is None else c
    order = sorted((e for e in range(n) if not out[e]), key=lambda e: (-key[e], e))[:top_k]
    ids, w = np.full(top_k, -1, dtype=np.int32), np.zeros(top_k)
    ids[: len(order)] = order
    if order:
        v = s[order]
        if renorm:
            if score == "sigmoid" and v.max() < 1e-200:  # the ratios of what underflows
                v = np.exp(z[order] - z[order].max())
            # (of a softmax that is the softmax over the chosen, also where all of theirs are 0)
            v = scores(z[order], score) if score == "softmax" else v / v.sum()
        w[: len(order)] = v * scale
    return ids, w


def route(z, bias, top_k, score, **kw):
    rows = [route_row(r, bias, top_k, score, **kw) for r in np.asarray(z, dtype=np.float64)]
    if not rows:
        return np.zeros((0, top_k), np.int32), np.zeros((0, top_k))
    return np.stack([r[0] for r in rows]), np.stack([r[1] for r in rows])
