"""Microscaled 4-bit floating point and the gated feed-forward block in float64 (test infrastructure only).

Written from the definitions: OCP Microscaling MXFP4 (32 columns share one power-of-two scale; elements
are E2M1) and H = act(X Wg^T) * (X Wu^T) with its derivatives. Shares no code with the GPU path.
"""
from __future__ import annotations

import math

import numpy as np

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def mx_quantize(x):
    """(codes, scales) of x (rows x cols): codes uint8 rows x 16 nblk, scales uint8 rows x nblk. Elements are
    matched by comparing distances to all eight magnitudes, ties going to the even code."""
    x = np.asarray(x, dtype=np.float64)
    rows, cols = x.shape
    nblk = -(-cols // 32)
    b = np.zeros((rows, nblk * 32))
    b[:, :cols] = x
    b = b.reshape(rows, nblk, 32)
    scales = np.zeros((rows, nblk), dtype=np.uint8)
    codes = np.zeros((rows, nblk, 32), dtype=np.uint8)
    mags = np.array(E2M1)
    for r in range(rows):
        for k in range(nblk):
            v = b[r, k]
            if not np.all(np.isfinite(v)):
                scales[r, k] = 255
                continue
            top = np.abs(v).max()
            e = -127 if top == 0.0 else max(-127, math.frexp(top)[1] - 3)
            scales[r, k] = e + 127
            m = np.abs(v) * 2.0 ** -e
            d = np.abs(m[:, None] - mags[None, :])
            near = d == d.min(axis=1, keepdims=True)
            best = np.where(near.sum(axis=1) == 2, np.argmax(near & (np.arange(8) % 2 == 0), axis=1), np.argmax(near, axis=1))
            codes[r, k] = best + 8 * np.signbit(v)
    return (codes[:, :, 0::2] | (codes[:, :, 1::2] << 4)).reshape(rows, nblk * 16), scales


def mx_values(codes, scales, cols):
    """The values of codes and scales, rows x cols (NaN where the scale is 255)."""
    codes, scales = np.asarray(codes), np.asarray(scales)
    rows, nblk = codes.shape[0], codes.shape[1] // 16
    c = np.stack((codes & 15, codes >> 4), axis=2).reshape(rows, nblk, 32)
    v = np.array(E2M1)[c & 7] * np.where(c & 8, -1.0, 1.0)
    s = scales[:, :nblk].astype(np.int64)
    sc = np.where(s == 255, np.nan, np.ldexp(1.0, s - 127))
    return (v * sc[:, :, None]).reshape(rows, nblk * 32)[:, :cols]


def act(a, kind):
    """(act(a), act'(a))."""
    a = np.asarray(a, dtype=np.float64)
    if kind == "silu":
        s = 1.0 / (1.0 + np.exp(-a))
        return a * s, s + a * s * (1.0 - s)
    if kind == "gelu":
        phi = 0.5 * (1.0 + np.vectorize(math.erf, otypes=[float])(a / math.sqrt(2.0)))
        return a * phi, phi + a * np.exp(-0.5 * a * a) / math.sqrt(2.0 * math.pi)
    if kind == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        t = np.tanh(c * (a + 0.044715 * a ** 3))
        return 0.5 * a * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * a * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * a * a)
    if kind == "relu":
        return np.where(a > 0, a, 0.0), np.where(a > 0, 1.0, 0.0)
    raise ValueError(kind)


def gated(X, Wg, Wu, kind):
    """(H, A, B)."""
    A, B = X @ Wg.T, X @ Wu.T
    return act(A, kind)[0] * B, A, B


def gated_grad(dH, A, B, X, Wg, Wu, kind):
    """(dA, dB, dX, dWg, dWu)."""
    f, df = act(A, kind)
    dA, dB = dH * B * df, dH * f
    return dA, dB, dA @ Wg + dB @ Wu, dA.T @ X, dB.T @ X
