"""Gated feed-forward layer and its gradients in plain numpy, 64 bits
(include/fconv_gated.h).  Shares no code with the kernels."""
from __future__ import annotations

import numpy as np
from scipy.special import erfc, expit


def act(g, name):
    """(act(g), act'(g))."""
    g = np.asarray(g, np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        if name == "silu":
            s, c = expit(g), expit(-g)
            return g * s, s + g * s * c
        if name == "gelu":
            cdf = 0.5 * erfc(-g / np.sqrt(2.0))
            return g * cdf, cdf + g * np.exp(-0.5 * g * g) / np.sqrt(2.0 * np.pi)
        if name == "gelu_tanh":
            v2 = 2.0 * np.sqrt(2.0 / np.pi) * (g + 0.044715 * g ** 3)
            s, c = expit(v2), expit(-v2)
            return g * s, s + g * s * c * 2.0 * np.sqrt(2.0 / np.pi) * (1.0 + 3.0 * 0.044715 * g * g)
        if name == "relu":
            return np.where(g > 0, g, np.where(np.isnan(g), g, 0.0)), np.where(np.isnan(g), g, (g > 0) * 1.0)
    raise ValueError(name)


def forward(x, w, name):
    """(y [T, F], g [T, F], u [T, F])."""
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    F = w.shape[0] // 2
    g, u = x @ w[:F].T, x @ w[F:].T
    return act(g, name)[0] * u, g, u


def backward(x, w, g, u, dy, name):
    """(dx [T, D], dw [2 F, D], [dg du] [T, 2 F])."""
    x, w, dy = (np.asarray(a, np.float64) for a in (x, w, dy))
    a, da = act(g, name)
    dz = np.concatenate((dy * u * da, dy * a), 1)
    return dz @ w, dz.T @ x, dz
