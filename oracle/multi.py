"""FP64 definition of one projection for the rows of many adapters.

Y[t, g] = X[t] W_g^T + bias_g + s_t (X[t] A_{a,g}^T) B_{a,g}^T with a = slot[t] and
s_t = scale[a] * row_scale[t] * request_scale; a slot outside the bank contributes nothing, and so
does a scale of exactly zero.
"""
from __future__ import annotations

import numpy as np


def row_scales(slot, scale, row_scale, request_scale):
    """s_t in float32 (the products are rounded one after another); 0 where no adapter is used."""
    f = np.float32
    slot = np.asarray(slot)
    ok = (slot >= 0) & (slot < len(scale))
    s = np.asarray(scale, f)[np.where(ok, slot, 0)]
    if row_scale is not None:
        s = (s * np.asarray(row_scale, f)).astype(f)
    s = (s * f(request_scale)).astype(f)
    return np.where(ok, s, f(0)).astype(np.float64)


def forward(X, W, bias, A, B, groups, slot, s, N):
    """(Y, S, E): the result, the magnitude sum |X||W|^T + |bias| + |s|(|X||A|^T)|B|^T of every
    element, and the adapters' part of it."""
    T = X.shape[0]
    Y = np.zeros((T, N)) if W is None else X @ W.T
    S = np.zeros((T, N)) if W is None else np.abs(X) @ np.abs(W).T
    E = np.zeros((T, N))
    if bias is not None:
        Y = Y + bias
        S = S + np.abs(bias)
    R, og = B.shape[2], N // groups
    for t in range(T):
        if s[t] == 0:
            continue
        a = slot[t]
        for g in range(groups):
            c = slice(g * og, (g + 1) * og)
            Ag, Bg = A[a, g * R:(g + 1) * R], B[a, c]
            Y[t, c] += s[t] * (X[t] @ Ag.T) @ Bg.T
            e = abs(s[t]) * (np.abs(X[t]) @ np.abs(Ag).T) @ np.abs(Bg).T
            S[t, c] += e
            E[t, c] += e
    return Y, S, E
