"""Grouped routing in fp64 (test infrastructure).

Scores s (softmax or sigmoid of the logits), choice values c = s + bias, the
groups_kept groups whose group_top largest choice values sum highest, in them
the k experts of largest c; ties to the lower id.  Weights are the scores of
the chosen experts, renormalised over them or not, times a scale.  Experts
whose logit or bias is NaN or at most -3.3e38 are masked: score 0 where the
logit masks, no part in a group's value, chosen last (lowest id first) and with
weight 0.  Plain sorts by (masked, -value, id) of every expert.
"""

from __future__ import annotations

import math

import numpy as np

LOWEST = -3.3e38
FLOAT_MAX = float(np.finfo(np.float32).max)


def _masked(v: float) -> bool:
    return math.isnan(v) or v <= LOWEST


def scores(row, score: str) -> list:
    z = [None if _masked(float(v)) else min(float(v), FLOAT_MAX) for v in row]
    if score == "sigmoid":
        # both branches are 1 / (1 + e^-z), without overflow
        return [0.0 if v is None else (1.0 / (1.0 + math.exp(-v)) if v >= -700 else math.exp(v)) for v in z]
    live = [v for v in z if v is not None]
    if not live:
        return [0.0] * len(z)
    top = max(live)
    e = [0.0 if v is None else math.exp(v - top) for v in z]
    total = math.fsum(e)
    return [v / total for v in e]


def route_grouped(logits, bias, k: int, score: str = "sigmoid", groups: int = 1, groups_kept: int = 1,
                  group_top: int = 2, renormalise: bool = True, scale: float = 1.0):
    """Returns (topk_idx int32 [T,k], topk_w float64 [T,k])."""
    T, E = logits.shape
    size = E // groups
    idx, w = np.zeros((T, k), np.int32), np.zeros((T, k))
    for t in range(T):
        s = scores(logits[t], score)
        off = [_masked(float(logits[t, e])) or (bias is not None and _masked(float(bias[e]))) for e in range(E)]
        c = [0.0 if off[e] else s[e] + (0.0 if bias is None else float(bias[e])) for e in range(E)]
        value = []
        for g in range(groups):
            best = sorted((c[e] for e in range(g * size, (g + 1) * size) if not off[e]), reverse=True)[:group_top]
            value.append((not best, -sum(best), g))
        kept = {g for _, _, g in sorted(value)[:groups_kept]}
        order = sorted((off[e], -c[e], e) for e in range(E) if e // size in kept)[:k]
        idx[t] = [e for _, _, e in order]
        w[t] = [0.0 if masked else s[e] for masked, _, e in order]
        total = math.fsum(w[t])
        if renormalise:
            w[t] = w[t] / total if total > 0 else 0.0
    return idx, w * scale
