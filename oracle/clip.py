"""Norm of gradients and clipping by it in plain numpy, 64 bits
(include/fconv_clip.h).  Shares no code with the kernels."""
from __future__ import annotations

import math

import numpy as np


def norm(grads):
    with np.errstate(over="ignore", invalid="ignore"):
        return math.sqrt(sum(float((np.asarray(g, np.float64) ** 2).sum()) for g in grads))


def clip(grads, max_norm, eps=1e-6, given=None):
    """(norm, clipped gradients)."""
    n = norm(grads) if given is None else given
    by = 1.0 if max_norm == math.inf else max_norm / (n + eps) if n + eps > 0 else math.inf if max_norm > 0 else math.nan
    by = 1.0 if by >= 1.0 else by
    with np.errstate(invalid="ignore"):
        return n, [by * np.asarray(g, np.float64) for g in grads]
