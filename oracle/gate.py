"""Gated routing, oracle side (test infrastructure): one token and one expert at a time, in fp64.

Scores are the softmax over all experts or a sigmoid each; the values that decide
the choice are the scores plus a bias; groups of consecutive experts are ranked by
their largest value or the sum of their two largest; ties go to the lower index;
a value that is -inf or NaN is never taken (id -1, weight 0).
"""
from __future__ import annotations

import math

import numpy as np


def scores(logits, sigmoid: bool) -> np.ndarray:
    l = np.asarray(logits, dtype=np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        if sigmoid:
            return 1.0 / (1.0 + np.exp(-l))
        z = np.exp(l - l.max(axis=-1, keepdims=True))
        return z / z.sum(axis=-1, keepdims=True)


def choose(s, K, select_bias=None, groups=1, group_topk=1, top2=False, renorm=True, scale=1.0):
    """One token: scores s [E] -> (ids [K], weights [K])."""
    E = len(s)
    c = [float(s[e]) + (float(select_bias[e]) if select_bias is not None else 0.0) for e in range(E)]
    c = [v if v > -math.inf else -math.inf for v in c]          # NaN: -inf
    if groups > 1:
        n = E // groups
        value = []
        for g in range(groups):
            best = sorted(c[g * n:(g + 1) * n], reverse=True)
            v = best[0] + best[1] if top2 else best[0]
            value.append(v if v > -math.inf else -math.inf)
        kept = sorted(range(groups), key=lambda g: (-value[g], g))[:group_topk]
        c = [v if e // n in kept else -math.inf for e, v in enumerate(c)]
    order = sorted(range(E), key=lambda e: (-c[e], e))[:K]
    ids = [e if c[e] > -math.inf else -1 for e in order]
    w = [float(s[e]) if e >= 0 else 0.0 for e in ids]
    if renorm:
        total = sum(w)
        w = [v / total if total > 0 else 0.0 for v in w]
    return ids, [v * scale for v in w]


def route(x, router_w, router_bias, K, sigmoid=False, **kw):
    """(ids int32 [T, K], weights fp64 [T, K], logits fp64 [T, E]) from exact fp64 copies of the inputs."""
    l = np.asarray(x, dtype=np.float64) @ np.asarray(router_w, dtype=np.float64).T
    if router_bias is not None:
        l = l + np.asarray(router_bias, dtype=np.float64)
    s = scores(l, sigmoid)
    ids = np.empty((len(l), K), dtype=np.int32)
    w = np.empty((len(l), K))
    for t in range(len(l)):
        ids[t], w[t] = choose(s[t], K, **kw)
    return ids, w, l
