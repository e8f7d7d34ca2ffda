"""Oracle of the 8-bit lm_head: e4m3 values with a scale for every 128 elements.

flashrec 0.1.0 (PyPI page), Features: W8A8 FP8, the RMS norm fused with the
quantisation. A block y shares scale = max(max |y|, 448 * 2^-100) / 448 and
stands for q * scale, q the e4m3 value nearest to y / scale (448: the largest).

The list of e4m3 values is made from the format's definition (sign, 4 exponent
bits with bias 7, 3 fraction bits, no infinities, 0x7f / 0xff NaN).

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).
"""
from __future__ import annotations

import numpy as np

BLOCK = 128
FP8_MAX = 448.0
MIN_AMAX = FP8_MAX * 2.0 ** -100


def e4m3_values() -> np.ndarray:
    """The value of each of the 256 e4m3 codes (NaN for 0x7f and 0xff)."""
    c = np.arange(256)
    e, f = (c >> 3) & 15, c & 7
    v = np.where(e == 0, f * 2.0 ** -9, (8 + f) * 2.0 ** (e - 10.0))
    v = np.where((c & 0x7F) == 0x7F, np.nan, v)
    return np.where(c >> 7, -v, v)


def blocks(y, rows: int):
    """Scales [ceil(M/rows), ceil(d/128)] of float64 y [M, d]."""
    M, d = y.shape
    out = np.empty((-(-M // rows), -(-d // BLOCK)))
    for i in range(out.shape[0]):
        for j in range(out.shape[1]):
            part = y[i * rows:(i + 1) * rows, j * BLOCK:(j + 1) * BLOCK]
            out[i, j] = max(np.abs(part).max(), MIN_AMAX) / FP8_MAX
    return out


def expand(scale, rows: int, shape):
    """A scale per element."""
    return np.repeat(np.repeat(scale, rows, 0)[:shape[0]], BLOCK, 1)[:, :shape[1]]


def residual_rmsnorm(x, residual, weight, eps):
    """(h, y) in float64."""
    h = x if residual is None else x + residual
    return h, h / np.sqrt((h * h).mean(1, keepdims=True) + eps) * weight


def lmhead_logits(hidden_codes, hidden_scale, w_codes, w_scale):
    """Logits [M, V] of uint8 e4m3 codes and their scales, and sum |h w|."""
    val = e4m3_values()
    h = val[hidden_codes] * expand(np.asarray(hidden_scale, np.float64), 1, hidden_codes.shape)
    w = val[w_codes] * expand(np.asarray(w_scale, np.float64), BLOCK, w_codes.shape)
    return h @ w.T, np.abs(h) @ np.abs(w).T
