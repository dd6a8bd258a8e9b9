"""A layer in 8 bits in 64 bits, straight from its formulas -- TEST INFRASTRUCTURE ONLY.

Arguments are float64 matrices (rows, depth) and vectors; q is int8 and scale float64.
"""
from __future__ import annotations

from fractions import Fraction

import numpy as np


def scale_of(top: float) -> float:
    """2^e with the smallest e from -126 to 121 for which top <= 127 * 2^e (exact: in rationals)."""
    e = -126
    top = Fraction(top)
    while e < 121 and top > 127 * Fraction(2) ** e:
        e += 1
    return 2.0 ** e


def quantize_rows(y):
    """(q, scale); a row that holds NaN or an infinity has scale NaN and q = 0."""
    q = np.zeros(y.shape, np.int8)
    scale = np.empty(y.shape[0])
    for r in range(y.shape[0]):
        if not np.isfinite(y[r]).all():
            scale[r] = np.nan
            continue
        scale[r] = scale_of(float(np.abs(y[r]).max()))
        q[r] = np.clip(np.rint(y[r] / scale[r]), -127, 127)      # to even at the half
    return q, scale


def rms_norm(h, weight, eps):
    """(y, rstd)."""
    r = 1.0 / np.sqrt(np.mean(h * h, axis=1) + eps)
    return h * r[:, None] * weight, r


def rms_norm_grad(h, weight, eps, dy, dh=None):
    """(dx, dweight)."""
    r = 1.0 / np.sqrt(np.mean(h * h, axis=1) + eps)
    xh = h * r[:, None]
    g = dy * weight
    dx = r[:, None] * (g - xh * np.mean(g * xh, axis=1, keepdims=True))
    return dx if dh is None else dx + dh, np.sum(dy * xh, axis=0)


def linear(xq, xs, wq, ws):
    whole = xq.astype(np.int64) @ wq.astype(np.int64).T
    return whole * xs[:, None] * ws


def linear_grad_input(dout, wq, ws):
    return dout @ (wq * ws[:, None])


def linear_grad_weight(dout, xq, xs):
    return dout.T @ (xq * xs[:, None])
