"""float64 oracle of the layer norm over the last dimension and its gradients.

TEST INFRASTRUCTURE ONLY (never imported by the product path).

    y = (x - mean) rstd w + b ,   rstd = 1 / sqrt(mean((x - mean)^2) + eps)

The backward is the chain rule written out: with x^ = (x - mean) rstd and g = dy w,
dx = rstd (g - mean(g) - x^ mean(g x^)), dw = sum over rows of dy x^, db = sum of dy.
"""
from __future__ import annotations

import numpy as np


def fwd(x, w=None, b=None, eps=1e-5):
    """(y, mean, rstd) for x [rows, d]."""
    x = np.asarray(x, np.float64)
    mean = x.mean(-1)
    c = x - mean[:, None]
    rstd = 1.0 / np.sqrt((c * c).mean(-1) + eps)
    y = c * rstd[:, None]
    if w is not None:
        y = y * np.asarray(w, np.float64)
    if b is not None:
        y = y + np.asarray(b, np.float64)
    return y, mean, rstd


def bwd(x, dy, mean, rstd, w=None):
    """(dx, dw, db) given the forward's statistics."""
    x, dy = np.asarray(x, np.float64), np.asarray(dy, np.float64)
    rstd = np.asarray(rstd, np.float64)[:, None]
    xh = (x - np.asarray(mean, np.float64)[:, None]) * rstd
    g = dy if w is None else dy * np.asarray(w, np.float64)
    dx = rstd * (g - g.mean(-1, keepdims=True) - xh * (g * xh).mean(-1, keepdims=True))
    return dx, (dy * xh).sum(0), dy.sum(0)
