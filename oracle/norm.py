"""Norms before and after a block with its gate and residual scale (oracle).

TEST INFRASTRUCTURE ONLY - see ``oracle/__init__.py``.  Float64 throughout;
``mq_norm`` in ``include/moe_quant.h`` states the formulas.
"""
from __future__ import annotations

import numpy as np


def rms_norm(v, weight, eps, offset):
    v = np.asarray(v, np.float64)
    mean = np.mean(v * v, axis=1, keepdims=True)
    return v / np.sqrt(mean + eps) * (offset + np.asarray(weight, np.float64))


def residual_update(x, residual, gate=None, post_weight=None, eps=1e-6, offset=0.0, scale=1.0):
    """(residual, scale * gate * z): the new residual is their sum, unrounded."""
    add = 0.0
    if x is not None:
        add = np.asarray(x, np.float64) if post_weight is None else rms_norm(x, post_weight, eps, offset)
        if gate is not None:
            add = add * np.asarray(gate, np.float64)
        add = add * scale
    r = np.zeros_like(add) if residual is None else np.asarray(residual, np.float64)
    return r, add + np.zeros_like(r)
