"""8-bit integers with a scale for each row, products grouped by expert, and norms in float64 (test infrastructure only).

Written from the definitions in include/kq.h. Shares no code with the GPU path.
"""
from __future__ import annotations

import numpy as np


def i8_quantize(x):
    """(codes int8, scales float32) of x (rows x cols): scale = a / 127 and m = 127 / a as fp32 values, codes the whole
    numbers nearest to the exact x m, ties to the even one."""
    x = np.asarray(x, dtype=np.float64)
    codes, scales = np.zeros(x.shape, dtype=np.int8), np.zeros(x.shape[0], dtype=np.float32)
    for r, row in enumerate(x):
        if not np.all(np.isfinite(row)):
            scales[r] = np.nan
            continue
        a = np.float32(np.abs(row).max())
        if a < np.float32(2.0 ** -119):
            continue
        scales[r] = a / np.float32(127)
        codes[r] = np.rint(row * np.float64(np.float32(127) / a))     # 24 + 24 bits: exact
    return codes, scales


def i8_values(codes, scales):
    """code * scale rounded to fp32."""
    return np.asarray(codes).astype(np.float32) * np.asarray(scales, dtype=np.float32)[:, None]


def spans(offsets, n):
    """(expert, first row, end) as any contents of the offsets are read: clamped to 0 .. n, raised to the largest before."""
    o = np.maximum.accumulate(np.clip(np.asarray(offsets, dtype=np.int64), 0, n))
    return [(k, int(o[k]), int(o[k + 1])) for k in range(len(o) - 1)]


def grouped(X, W, offsets):
    """(Y, rows that belong to an expert): Y_r = X_r W_k^T, zero elsewhere."""
    Y, inside = np.zeros((X.shape[0], W.shape[1])), np.zeros(X.shape[0], dtype=bool)
    for k, a, b in spans(offsets, X.shape[0]):
        Y[a:b] = X[a:b] @ W[k].T
        inside[a:b] = True
    return Y, inside


def grouped_grad(dY, X, W, offsets):
    """(dX, dW) of the sum of grouped(X, W) * dY."""
    dX, dW = np.zeros(X.shape), np.zeros(W.shape)
    for k, a, b in spans(offsets, X.shape[0]):
        for r in range(a, b):
            dX[r] = dY[r] @ W[k]
        dW[k] = dY[a:b].T @ X[a:b]
    return dX, dW


def norm(X, gamma, beta, kind, eps):
    """(Y, mean, 1 / deviation)."""
    m = X.mean(axis=1) if kind == "layer" else np.zeros(X.shape[0])
    t = X - m[:, None]
    r = 1.0 / np.sqrt((t * t).mean(axis=1) + eps)
    return t * r[:, None] * gamma + beta, m, r


def norm_grad(dY, X, gamma, mean, rstd, kind):
    """(dX, dgamma, dbeta)."""
    h = (X - mean[:, None]) * rstd[:, None]
    g = dY * gamma
    dX = g - h * (g * h).mean(axis=1, keepdims=True)
    if kind == "layer":
        dX = dX - g.mean(axis=1, keepdims=True)
    return dX * rstd[:, None], (dY * h).sum(axis=0), dY.sum(axis=0)
