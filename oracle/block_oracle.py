"""fp64 oracle of the operators around the expert layer (test infrastructure, like the rest of this package):
residual addition with RMS norm and its backward, the router's balance and z losses with their gradient, and the
router's products for an additional logit gradient.  Plain numpy, from the definitions."""
from __future__ import annotations

import numpy as np


def rmsnorm(h, weight, eps):
    """(y, rstd) of the rows of h."""
    h = np.asarray(h, dtype=np.float64)
    rstd = 1.0 / np.sqrt(np.mean(h * h, axis=1) + eps)
    return h * rstd[:, None] * np.asarray(weight, dtype=np.float64), rstd


def rmsnorm_backward(dy, h, weight, rstd, dh=None):
    """(gradient of h, gradient of the weight) for an upstream gradient dy of y and dh of h."""
    dy, h, w = (np.asarray(a, dtype=np.float64) for a in (dy, h, weight))
    xhat = h * np.asarray(rstd, dtype=np.float64)[:, None]
    g = dy * w
    out = np.asarray(rstd, dtype=np.float64)[:, None] * (g - xhat * np.mean(g * xhat, axis=1, keepdims=True))
    if dh is not None:
        out = out + np.asarray(dh, dtype=np.float64)
    return out, np.sum(dy * xhat, axis=0)


def softmax_rows(logits):
    """(softmax, log-sum-exp) of every row; zeros for a row without a finite logit."""
    m = logits.max(axis=1, keepdims=True) if logits.shape[1] else np.zeros((len(logits), 1))
    dead = np.isneginf(m)
    m = np.where(dead, 0.0, m)
    ex = np.exp(logits - m)
    z = ex.sum(axis=1, keepdims=True)
    p = np.where(dead, 0.0, ex / np.where(dead, 1.0, z))
    return p, np.where(dead, 0.0, m + np.log(np.where(dead, 1.0, z)))[:, 0]


def balance_loss(logits, topk_ids, balance_coef, z_coef, mask=None, seq_offsets=None, dloss=1.0):
    """dict(loss [3], counts [B, E], probs [B, E], dlogits [T, E])."""
    logits = np.asarray(logits, dtype=np.float64)
    T, E = logits.shape
    K = topk_ids.shape[1]
    cuts = [0, T] if seq_offsets is None else list(seq_offsets)
    keep = np.ones(T, dtype=bool) if mask is None else np.asarray(mask).astype(bool)
    p, lse = softmax_rows(logits)
    B = len(cuts) - 1
    counts, probs = np.zeros((B, E), dtype=np.int64), np.zeros((B, E))
    dp = np.zeros((T, E))  # the balance loss's gradient of p, before the coefficients
    balance, used = 0.0, 0
    for b in range(B):
        rows = [t for t in range(cuts[b], cuts[b + 1]) if keep[t]]
        if not rows:
            continue
        used += 1
        counts[b] = np.bincount(topk_ids[rows].reshape(-1), minlength=E)
        probs[b] = p[rows].mean(axis=0)
        f = counts[b] * (E / (K * len(rows)))
        balance += float(np.dot(f, probs[b]))
        dp[rows] = f / len(rows)
    n = int(keep.sum())
    if used:
        balance, dp = balance / used, dp / used
    z = float(np.mean(lse[keep] ** 2)) if n else 0.0
    g = balance_coef * p * (dp - np.sum(p * dp, axis=1, keepdims=True))
    if n:
        g = g + (2.0 * z_coef / n) * lse[:, None] * p * keep[:, None]
    return dict(loss=np.array([balance_coef * balance + z_coef * z, balance, z]), counts=counts, probs=probs,
                dlogits=dloss * g)


def router_backward(dlogits, X, W_r, dX_in=None, dW_r_in=None):
    """(dX, dW_r) with the given gradients added."""
    dl, X, W = (np.asarray(a, dtype=np.float64) for a in (dlogits, X, W_r))
    dX, dW = dl @ W.T, X.T @ dl
    return (dX if dX_in is None else dX + dX_in), (dW if dW_r_in is None else dW + dW_r_in)
