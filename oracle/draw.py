"""The definition of a draw in 64 bits (test infrastructure; shares nothing with the library)."""
from __future__ import annotations

import math

import numpy as np


def draw(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(id, probability, margin) of one row: the token drawn, and how far the decisions that led to it were from
    falling otherwise, relative to the weights that they compare."""
    l = np.asarray(logits, dtype=np.float64)
    V = l.size
    if np.isnan(l).any() or np.isposinf(l).any():
        return 0, math.nan, math.inf
    M = l.max()
    if np.isneginf(M):
        return 0, 0.0, math.inf
    if not temperature > 0:
        return int(np.argmax(l)), 1.0, math.inf
    with np.errstate(over="ignore", invalid="ignore"):
        z = (M - l) / temperature
    w = np.where(np.isneginf(l), 0.0, np.exp(-np.where(np.isnan(z), 0.0, z)))
    order = np.lexsort((np.arange(V), -l))  # by falling logits, then by id
    margin = math.inf
    if 0 < top_k < V:
        order = order[:top_k]
    if top_p < 1.0:
        ws = w[order]
        before = np.concatenate([[0.0], np.cumsum(ws)[:-1]])
        want = max(top_p, 0.0) * ws.sum()
        stay = before < want
        stay[0] = True
        near = np.abs(before[1:] - want)
        # (a token without weight may stay or not)
        if near.size and want > 0:
            margin = min(margin, near[ws[1:] > 0].min(initial=math.inf) / ws.sum())
        order = order[stay]
    if min_p > 0:
        least = min(min_p, 1.0)
        ws = w[order]
        differ = np.abs(ws - least) / least
        margin = min(margin, differ[ws != 1.0].min(initial=math.inf))
        order = order[(ws >= least) | (np.arange(ws.size) == 0)]
    ids = np.sort(order)
    ids = ids[w[ids] > 0]
    upto = np.cumsum(w[ids])
    f = 0.0 if not u > 0 else min(float(u), 1.0)
    target = f * upto[-1]
    at = min(int((upto <= target).sum()), ids.size - 1)
    if f < 1.0 and f > 0.0:
        margin = min(margin, np.abs(upto[:-1] - target).min(initial=math.inf) / upto[-1])
    return int(ids[at]), float(w[ids[at]] / upto[-1]), margin
