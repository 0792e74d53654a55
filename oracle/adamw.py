"""AdamW (decoupled weight decay) in FP64, and the 8-bit blocks its moments may be held in.

A block is 256 consecutive elements with one scale a (their largest magnitude).  A code q stands
for a sign(q) (|q| / 127)^2 (signed, first moments) or a (q / 255)^4 (unsigned, second moments).
The codes are defined by the float32 sequence: divide by the scale, root (twice for the unsigned
form), multiply by the largest code, round half to even, each step correctly rounded; an unsigned
value above zero is never coded as zero.  A code's share u of the largest code is the rounded product of
the code and the rounded reciprocal of the largest code; the value is u |u| a or (u u)(u u) a, each
product rounded.
"""
from __future__ import annotations

import numpy as np

BLOCK = 256
f32 = np.float32


def step(p, g, m, v, lr, beta1, beta2, eps, wd, t, grad_scale=1.0):
    """(p, m, v) after one step, in FP64."""
    p, g, m, v = (np.asarray(a, dtype=np.float64) for a in (p, g, m, v))
    g = g * grad_scale
    m = beta1 * m + (1.0 - beta1) * g
    v = beta2 * v + (1.0 - beta2) * g * g
    with np.errstate(all="ignore"):
        den = np.sqrt(v) / np.sqrt(1.0 - beta2 ** t) + eps
        p = p * (1.0 - lr * wd) - lr / (1.0 - beta1 ** t) * (m / den)
    return p, m, v


def moments_f32(g, m, v, beta1, beta2, grad_scale):
    """The moments' float32 sequence: every product and sum rounded by itself."""
    g = (np.asarray(g, f32) * f32(grad_scale)).astype(f32)
    m = (f32(beta1) * m).astype(f32) + (f32(1.0 - beta1) * g).astype(f32)
    v = (f32(beta2) * v).astype(f32) + (f32(1.0 - beta2) * (g * g).astype(f32)).astype(f32)
    return m.astype(f32), v.astype(f32)


def _blocks(x):
    n = x.size
    out = np.zeros((n + BLOCK - 1) // BLOCK * BLOCK, dtype=x.dtype)
    out[:n] = x.reshape(-1)
    return out.reshape(-1, BLOCK)


def encode(x, signed):
    """(codes [n], absmax) of float32 values, by the float32 sequence."""
    b = _blocks(np.asarray(x, dtype=f32))
    top = np.abs(b).max(axis=1)
    with np.errstate(all="ignore"):
        s = np.sqrt(np.where(top[:, None] > 0, np.abs(b) / top[:, None], f32(0)).astype(f32))
        q = (f32(127) * s) if signed else (f32(255) * np.sqrt(s))
        q = np.rint(q.astype(f32))
    q = np.nan_to_num(q, nan=0.0)
    if signed:
        q = np.where(b < 0, -q, q).astype(np.int8)
    else:
        q = np.where((b > 0) & (q < 1), 1, q).astype(np.uint8)
    return q.reshape(-1)[:x.size], top


def decode(q, top, signed):
    """float32 values of codes, by the float32 sequence."""
    b = _blocks(np.asarray(q).astype(f32))
    u = (b * (f32(1) / f32(127 if signed else 255))).astype(f32)
    u = (u * np.abs(u)).astype(f32) if signed else ((u * u).astype(f32) * (u * u).astype(f32)).astype(f32)
    with np.errstate(all="ignore"):
        return (u * top[:, None]).astype(f32).reshape(-1)[:np.asarray(q).size]
