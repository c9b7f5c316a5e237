"""Float64 reference of the low-rank adapters and their gradients (test infrastructure only).

One request at a time, from the definition.  It shares no code with the HIP path.
"""
from __future__ import annotations

import numpy as np


def requests(adapter, start, n, T):
    """(lo, hi, adapter) of every request with rows; adapter -1: none, -2: an id that does not exist."""
    for i, a in enumerate(adapter):
        lo, hi = max(int(start[i]), 0), min(int(start[i + 1]), T)
        if hi > lo:
            yield lo, hi, (int(a) if 0 <= a < n else -1 if a < 0 else -2)


def factors(A, B, scale, rank, a):
    r = A.shape[1] if rank is None else min(max(int(rank[a]), 0), A.shape[1])
    return float(scale[a]), A[a, :r].astype(np.float64), B[a, :, :r].astype(np.float64)


def forward(x, A, B, adapter, start, scale, rank, base):
    """(y, magnitude of the sums behind each element, rows written): y = base + s (x A^T) B^T."""
    T, N = x.shape[0], B.shape[1]
    y = np.zeros((T, N)) if base is None else base.astype(np.float64).copy()
    mag = np.zeros((T, N))
    written = np.zeros(T, dtype=bool)
    for lo, hi, a in requests(adapter, start, A.shape[0], T):
        written[lo:hi] = True
        if a == -2:
            y[lo:hi] = np.nan
        elif a >= 0:
            s, down, up = factors(A, B, scale, rank, a)
            y[lo:hi] += s * (x[lo:hi] @ down.T) @ up.T
            mag[lo:hi] = abs(s) * (np.abs(x[lo:hi]) @ np.abs(down).T) @ np.abs(up).T
    return y, mag, written


def backward(dy, x, A, B, adapter, start, scale, rank, base):
    """((dx, dA, dB), their magnitudes, rows of dx written)."""
    T, H = x.shape
    dx = np.zeros((T, H)) if base is None else base.astype(np.float64).copy()
    dA, dB = np.zeros(A.shape), np.zeros(B.shape)
    mx, mA, mB = np.zeros((T, H)), np.zeros(A.shape), np.zeros(B.shape)
    written = np.zeros(T, dtype=bool)
    for lo, hi, a in requests(adapter, start, A.shape[0], T):
        written[lo:hi] = True
        if a == -2:
            dx[lo:hi] = np.nan
        elif a >= 0:
            s, down, up = factors(A, B, scale, rank, a)
            k = down.shape[0]
            d, xs = dy[lo:hi].astype(np.float64), x[lo:hi].astype(np.float64)
            u, v = s * xs @ down.T, s * d @ up
            dx[lo:hi] += v @ down
            dA[a, :k] += v.T @ xs
            dB[a, :, :k] += d.T @ u
            mu = abs(s) * np.abs(xs) @ np.abs(down).T
            mv = abs(s) * np.abs(d) @ np.abs(up)
            mx[lo:hi] = mv @ np.abs(down)
            mA[a, :k] += mv.T @ np.abs(xs)
            mB[a, :, :k] += np.abs(d).T @ mu
    return (dx, dA, dB), (mx, mA, mB), written
