"""Queries and keys before attention, and attention of one token over a paged
cache (oracle).

TEST INFRASTRUCTURE ONLY - see ``oracle/__init__.py``.  Float64 throughout;
``mq_rotary`` and ``moe_quant_attend`` in ``include/moe_quant.h`` state the
formulas.
"""
from __future__ import annotations

import numpy as np


def turn(x, weight, eps, angles, interleaved):
    """Heads ``x`` [T, H, D] normed (``weight`` [D] or None) and rotated by the
    cosines and sines ``angles`` [T, R] (None: not at all)."""
    x = np.asarray(x, np.float64)
    if weight is not None:
        x = x / np.sqrt((x * x).mean(2, keepdims=True) + eps) * np.asarray(weight, np.float64)
    if angles is None:
        return x
    half = angles.shape[1] // 2
    y = x.copy()
    for i in range(half):
        one, two = (2 * i, 2 * i + 1) if interleaved else (i, half + i)
        c, s = angles[:, i, None].astype(np.float64), angles[:, half + i, None].astype(np.float64)
        y[:, :, one] = x[:, :, one] * c - x[:, :, two] * s
        y[:, :, two] = x[:, :, two] * c + x[:, :, one] * s
    return y


def attend(q, k, v, table, lengths, scale, window=0):
    """(out [B, Hq, D], lse [B, Hq], spread [B, Hq, D], reach [B, Hq]): spread is the
    sum of p |v|, reach the largest scale * sum |q k| of a token.  ``k`` and ``v``
    [pages, Hk, page, D] hold the values the cache stands for."""
    q = np.asarray(q, np.float64)
    b, hq, d = q.shape
    pages, hk, page, _ = k.shape
    out, spread = np.zeros((b, hq, d)), np.zeros((b, hq, d))
    lse, reach = np.full((b, hq), -np.inf), np.zeros((b, hq))
    for i in range(b):
        n = max(0, min(int(lengths[i]), table.shape[1] * page))
        at = [j for j in range(max(0, n - window) if window else 0, n) if 0 <= table[i, j // page] < pages]
        if not at:
            continue
        at = np.array(at)
        p, s = table[i, at // page], at % page
        for h in range(hq):
            kk, vv = k[p, h // (hq // hk), s].astype(np.float64), v[p, h // (hq // hk), s].astype(np.float64)
            score = scale * (kk @ q[i, h])
            top = score.max()
            e = np.exp(score - top)
            lse[i, h] = top + np.log(e.sum())
            e /= e.sum()
            out[i, h], spread[i, h] = e @ vv, e @ np.abs(vv)
            reach[i, h] = abs(scale) * (np.abs(kk) @ np.abs(q[i, h])).max()
    return out, lse, spread, reach
