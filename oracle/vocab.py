"""Losses over vocabulary rows in 64 bits, straight from their formulas -- TEST INFRASTRUCTURE ONLY.

`x` is a float64 matrix of logits (rows, vocab), `it` the factor 1 / temperature. z = x * it,
p = softmax(z) of each row; a row with nothing but -inf has no distribution.
"""
from __future__ import annotations

import numpy as np


def _order(row):
    """Indices by value, largest first: NaN, then +inf, ..., ties to the lower index."""
    key = np.where(np.isnan(row), np.inf, row)
    return sorted(range(row.size), key=lambda v: (0 if np.isnan(row[v]) else 1, -key[v], v))


def log_softmax(x, it):
    z = x.astype(np.float64) * it
    out = np.full(z.shape, -np.inf)
    for r in range(z.shape[0]):
        m = np.max(z[r]) if z.shape[1] else -np.inf
        if np.isneginf(m):
            continue
        if np.isnan(z[r]).any() or np.isposinf(m):
            out[r] = np.nan
            continue
        out[r] = (z[r] - m) - np.log(np.sum(np.exp(z[r] - m)))
    return out


def _xlogx(p, lp):
    return np.where(p > 0, p * np.where(p > 0, lp, 0.0), np.where(np.isnan(p), np.nan, 0.0))


def token_logprobs(x, it, targets=None, top_k=0):
    """(logprob, entropy, top_idx, top_logprob)."""
    lp = log_softmax(x, it)
    p = np.exp(lp)
    logprob = None
    if targets is not None:
        logprob = np.array([0.0 if t < 0 else lp[r, t] for r, t in enumerate(targets)])
    entropy = -_xlogx(p, lp).sum(1)
    idx = np.full((x.shape[0], top_k), -1, np.int32)
    val = np.full((x.shape[0], top_k), -np.inf)
    for r in range(x.shape[0]):
        if top_k:
            order = [v for v in _order(x[r].astype(np.float64)) if not np.isneginf(x[r, v])][:top_k]
            idx[r, :len(order)] = order
            val[r, :len(order)] = lp[r, order]
    return logprob, entropy, idx, val


def token_logprobs_grad(x, it, targets=None, g=None, h=None, top_idx=None, g_top=None):
    """Gradient of sum(g logprob) + sum(h entropy) + sum(g_top top_logprob) by x."""
    lp = log_softmax(x, it)
    p = np.exp(lp)
    entropy = -_xlogx(p, lp).sum(1)
    out = np.zeros(x.shape)
    for r in range(x.shape[0]):
        if np.isneginf(lp[r]).all():
            continue
        if g is not None and targets[r] >= 0:
            out[r] -= g[r] * p[r]
            out[r, targets[r]] += g[r]
        if h is not None:
            out[r] -= h[r] * (_xlogx(p[r], lp[r]) + p[r] * entropy[r])
        if g_top is not None:
            for i, w in zip(top_idx[r], g_top[r]):
                if i >= 0:
                    out[r] -= w * p[r]
                    out[r, i] += w
    return out * it


def teacher(idx, val, it, tail):
    """(log q, q) of the lists; absent entries have q = 0."""
    v = np.where(idx >= 0, val.astype(np.float64), -np.inf)
    if tail:
        return v, np.exp(v)
    lq = np.full(v.shape, -np.inf)
    for r in range(v.shape[0]):
        m = v[r].max() if v.shape[1] else -np.inf
        if not np.isneginf(m):
            z = (v[r] - m) * it
            lq[r] = z - np.log(np.exp(z).sum())
    return lq, np.exp(lq)


def distill(x, it, idx, val, tail):
    """Loss of each row."""
    lp = log_softmax(x, it)
    lq, q = teacher(idx, val, it, tail)
    loss = np.zeros(x.shape[0])
    for r in range(x.shape[0]):
        for j in range(idx.shape[1]):
            if q[r, j] > 0:
                loss[r] += q[r, j] * (lq[r, j] - lp[r, idx[r, j]])
        if tail:
            rho = max(0.0, 1.0 - q[r].sum())
            log_r = _log_rest(lp[r], idx[r])
            if rho > 0 and not np.isneginf(log_r):
                loss[r] += rho * (np.log(rho) - log_r)
    return loss


def _log_rest(lp, idx):
    outside = np.ones(lp.size, bool)
    outside[idx[idx >= 0]] = False
    rest = lp[outside]
    m = rest.max() if rest.size else -np.inf
    return m if np.isneginf(m) else m + np.log(np.exp(rest - m).sum())


def distill_grad(x, it, idx, val, tail, g):
    lp = log_softmax(x, it)
    p = np.exp(lp)
    _, q = teacher(idx, val, it, tail)
    out = np.zeros(x.shape)
    for r in range(x.shape[0]):
        if np.isneginf(lp[r]).all():
            continue
        mass = q[r].sum()
        out[r] = mass * p[r]
        if tail:
            rho = max(0.0, 1.0 - mass)
            log_r = _log_rest(lp[r], idx[r])
            if not np.isneginf(log_r):
                outside = np.ones(x.shape[1], bool)
                outside[idx[r][idx[r] >= 0]] = False
                # p / R outside is a softmax of its own: from log p it would lose its digits where R is next to nothing
                share = np.exp(log_softmax(np.where(outside, x[r], -np.inf)[None], it)[0])
                out[r] += rho * p[r] - rho * share
        for j in range(idx.shape[1]):
            if idx[r, j] >= 0:
                out[r, idx[r, j]] -= q[r, j]
        out[r] *= g[r] * it
    return out
