"""FP64 definition of layer norm and the form without a mean, forward and backward.

y = (x - mu) r w + b with r = 1 / sqrt(var + eps); without a mean mu = 0 and var is the mean
square.  The backward follows from the chain rule with xh = (x - mu) r and h = dy w:
dx = r (h - mean(h) - xh mean(h xh)) (no mean(h) without a mean), dw = sum dy xh, db = sum dy.
"""
from __future__ import annotations

import numpy as np


def forward(x, w=None, b=None, eps=1e-5, layer=True):
    """(y, mu, r) of every row."""
    x = np.asarray(x, dtype=np.float64)
    mu = x.mean(axis=1) if layer else np.zeros(x.shape[0])
    d = x - mu[:, None]
    with np.errstate(all="ignore"):
        r = 1.0 / np.sqrt((d * d).mean(axis=1) + eps)
        y = d * r[:, None]
        if w is not None:
            y = y * w
        if b is not None:
            y = y + b
    return y, mu, r


def backward(dy, x, w, mu, r, layer=True):
    """(dx, dw, db) from the saved mu and r."""
    dy, x = np.asarray(dy, dtype=np.float64), np.asarray(x, dtype=np.float64)
    xh = (x - mu[:, None]) * r[:, None]
    h = dy if w is None else dy * w
    dx = h - xh * (h * xh).mean(axis=1, keepdims=True)
    if layer:
        dx = dx - h.mean(axis=1, keepdims=True)
    return dx * r[:, None], (dy * xh).sum(axis=0), dy.sum(axis=0)
