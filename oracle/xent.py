"""Linear softmax cross entropy and its gradient in plain numpy, 64 bits
(include/fconv_xent.h).  Shares no code with the kernels."""
from __future__ import annotations

import numpy as np


def forward(h, w, target, ignore_index=-100):
    """(loss [T], lse [T], logits [T, V])."""
    h, w = np.asarray(h, np.float64), np.asarray(w, np.float64)
    T, V = h.shape[0], w.shape[0]
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        z = h @ w.T
        m = z.max(1)
        safe = np.where(np.isfinite(m), m, 0.0)
        lse = safe + np.log(np.exp(z - safe[:, None]).sum(1))
        lse = np.where(np.isnan(z).any(1), np.nan, lse)
        loss = np.full(T, np.nan)
        ok = (target >= 0) & (target < V)
        rows = np.arange(T)[ok]
        loss[rows] = lse[rows] - z[rows, target[rows]]
    loss[target == ignore_index] = 0.0
    return loss, lse, z


def logit_gradient(z, lse, target, dloss, ignore_index=-100):
    """g [T, V]."""
    with np.errstate(invalid="ignore", over="ignore"):
        g = np.exp(z - lse[:, None])
    T, V = z.shape
    ok = (target >= 0) & (target < V)
    g[np.arange(T)[ok], target[ok]] -= 1.0
    g[~ok] = np.nan
    g *= np.asarray(dloss, np.float64)[:, None]
    g[target == ignore_index] = 0.0
    return g


def backward(h, w, target, lse, dloss, ignore_index=-100):
    """(dh [T, D], dw [V, D], g [T, V])."""
    h, w = np.asarray(h, np.float64), np.asarray(w, np.float64)
    g = logit_gradient(h @ w.T, lse, target, dloss, ignore_index)
    keep = target != ignore_index  # an ignored token's h does not matter
    return g @ w, g[keep].T @ h[keep], g
