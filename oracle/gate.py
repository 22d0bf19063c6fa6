"""Gated routing: scores, balance bias, groups, top-k, weights (oracle).

TEST INFRASTRUCTURE ONLY - see ``oracle/__init__.py``.

A plain loop over the tokens in float64 of what ``mq_gate`` in
``include/moe_quant.h`` states.
"""
from __future__ import annotations

import math

import numpy as np


def _sigmoid(v: float) -> float:
    if v >= 0:
        return 1.0 / (1.0 + math.exp(-v))
    e = math.exp(v)
    return e / (1.0 + e)


def gate(logits, k, score="softmax", bias=None, groups=1, topk_groups=1, group_top=1,
         renormalize=True, scale=1.0):
    """ids int32 [T, k] and weights float64 [T, k] of ``logits`` [T, E]."""
    logits = np.asarray(logits, dtype=np.float64)
    t, e = logits.shape
    per = e // groups
    ids, weights = np.zeros((t, k), np.int32), np.zeros((t, k))
    biggest = float(np.finfo(np.float32).max)
    for r in range(t):
        x = [-math.inf if math.isnan(v) else min(float(v), biggest) for v in logits[r]]
        top = max(x)
        if score == "sigmoid":
            s = [0.0 if v == -math.inf else _sigmoid(v) for v in x]
            # log sigmoid, for renormalised weights of very negative logits
            logs = [-math.inf if v == -math.inf else min(v, 0.0) - math.log1p(math.exp(-abs(v))) for v in x]
        else:
            p = [0.0 if v == -math.inf else math.exp(v - top) for v in x]
            z = math.fsum(p)
            s = [v / z if z else 0.0 for v in p]
            logs = x
        live = [v > -math.inf for v in x]
        c = list(s)
        if bias is not None:
            for i in range(e):
                b = min(float(bias[i]), biggest)
                live[i] = live[i] and b > -math.inf          # False for NaN too
                c[i] = s[i] + b
        # without a bias the scores' order is the logits' own
        order = x if bias is None else c
        order = [order[i] if live[i] else -math.inf for i in range(e)]
        c = [c[i] if live[i] else -math.inf for i in range(e)]
        allowed = list(range(e))
        if groups > 1:
            def group_score(g):
                # the largest one in the logits' order where that is the order
                best = sorted((c if group_top == 2 else order)[g * per:(g + 1) * per], reverse=True)
                return best[0] if group_top == 1 else best[0] + best[1]
            ranked = sorted(range(groups), key=lambda g: (-group_score(g), g))[:topk_groups]
            allowed = [i for i in range(e) if i // per in ranked]
        chosen = sorted(allowed, key=lambda i: (-order[i], i))[:k]
        if renormalize:
            m = max(logs[i] if live[i] else -math.inf for i in chosen)
            w = [math.exp(logs[i] - m) if live[i] else 0.0 for i in chosen]
            total = math.fsum(w)
            w = [v / total if total else 0.0 for v in w]
        else:
            w = [s[i] if live[i] else 0.0 for i in chosen]
        ids[r], weights[r] = chosen, [v * scale for v in w]
    return ids, weights
