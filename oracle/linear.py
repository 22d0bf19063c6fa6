"""The dense product on E4M3 weights with a scale per block of 128 (oracle).

TEST INFRASTRUCTURE ONLY - see ``oracle/__init__.py``.  Float64, but for the
quantization of the rows, which ``mq_linear`` in ``include/moe_quant.h`` defines
by one FP32 product and one FP32 division.
"""
from __future__ import annotations

import numpy as np

from . import codecs


def quantize_rows(x):
    """(codes uint8 [T, 128 G], scales float32 [T, G]) of rows [T, K] of FP32
    numbers, the last block filled up by zeros."""
    x = np.asarray(x, np.float32)
    t, k = x.shape
    g = -(-k // 128)
    v = np.zeros((t, g * 128), np.float32)
    v[:, :k] = x
    v = v.reshape(t, g, 128)
    u = np.abs(v).max(2) * (np.float32(1.0) / np.float32(codecs.E4M3_MAX))
    s = np.where(u > 0, u, np.float32(1.0)).astype(np.float32)
    q = (v / s[:, :, None]).astype(np.float32)
    return codecs.quantize_e4m3(q.astype(np.float64)).reshape(t, g * 128), s


def forward(x, w, scale, residual=None):
    """(y, sum of the terms' magnitudes, sum over the blocks of each one's largest
    term), all [T, N]: y unrounded."""
    codes, s = quantize_rows(x)
    t, k = np.shape(x)
    a = codecs.decode_e4m3(codes) * np.repeat(s.astype(np.float64), 128, 1)
    n = w.shape[0]
    wide = np.repeat(np.repeat(np.asarray(scale, np.float64), 128, 0)[:n], 128, 1)[:, :k]
    v = codecs.decode_e4m3(w) * wide
    y, size = a[:, :k] @ v.T, np.abs(a[:, :k]) @ np.abs(v).T
    if residual is not None:
        y, size = y + np.asarray(residual, np.float64), size + np.abs(np.asarray(residual, np.float64))
    largest = np.zeros_like(y)
    for at in range(0, k, 128):
        block, wide = np.abs(a[:, at:min(k, at + 128)]), np.abs(v[:, at:at + 128])
        for i in range(t):
            largest[i] += (wide * block[i]).max(1)
    return y, size, largest
