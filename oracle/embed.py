"""Embedding lookup and its gradient in plain numpy, 64 bits
(include/fconv_embed.h).  Shares no code with the kernels."""
from __future__ import annotations

import numpy as np


def forward(w, token, scale=1.0, ignore_index=-100):
    """y [T, D]."""
    w, token = np.asarray(w, np.float64), np.asarray(token)
    y = np.full((len(token), w.shape[1]), np.nan)
    ok = (token >= 0) & (token < w.shape[0])
    y[ok] = float(np.float32(scale)) * w[token[ok]]
    y[token == ignore_index] = 0.0
    return y


def backward(token, dy, V, scale=1.0, ignore_index=-100):
    """dw [V, D]."""
    dy, token = np.asarray(dy, np.float64), np.asarray(token)
    dw = np.zeros((V, dy.shape[1]))
    ok = (token >= 0) & (token < V) & (token != ignore_index)
    np.add.at(dw, token[ok], dy[ok])
    return float(np.float32(scale)) * dw
