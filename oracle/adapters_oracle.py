"""Plain fp64 CPU reference of the low-rank adapters, the input gradients of low-bit
projections and the ragged 16-bit expert products (test infrastructure only).

All arguments are numpy arrays holding the values themselves (fp64, or anything that
converts exactly)."""
from __future__ import annotations

import numpy as np


def _f64(x):
    return np.asarray(x, dtype=np.float64)


def adapter_rows(ids, L):
    """(a, rows) of every adapter with rows; ids outside [0, L) have none."""
    ids = np.asarray(ids)
    for a in range(L):
        rows = np.nonzero(ids == a)[0]
        if len(rows):
            yield a, rows


def lora_t(X, A, ids):
    """T[m] = A[a] x_m (zeros without an adapter)."""
    X, A = _f64(X), _f64(A)
    T = np.zeros((X.shape[0], A.shape[1]))
    for a, rows in adapter_rows(ids, A.shape[0]):
        T[rows] = X[rows] @ A[a].T
    return T


def lora_add(X, A, B, ids, scale=None, base=None):
    """Y[m] = base[m] + s_a B[a] (A[a] x_m)."""
    B = _f64(B)
    T = lora_t(X, A, ids)
    Y = np.zeros((T.shape[0], B.shape[1])) if base is None else _f64(base).copy()
    for a, rows in adapter_rows(ids, B.shape[0]):
        s = 1.0 if scale is None else float(scale[a])
        Y[rows] += s * (T[rows] @ B[a].T)
    return Y


def lora_grad(dY, X, A, B, ids, scale=None, T=None, base=None):
    """(dX, dA, dB) of lora_add."""
    dY, X, A, B = _f64(dY), _f64(X), _f64(A), _f64(B)
    T = lora_t(X, A, ids) if T is None else _f64(T)
    dX = np.zeros(X.shape) if base is None else _f64(base).copy()
    dA, dB = np.zeros(A.shape), np.zeros(B.shape)
    for a, rows in adapter_rows(ids, A.shape[0]):
        s = 1.0 if scale is None else float(scale[a])
        dT = s * (dY[rows] @ B[a])
        dX[rows] += dT @ A[a]
        dA[a] = dT.T @ X[rows]
        dB[a] = s * (dY[rows].T @ T[rows])
    return dX, dA, dB


def grouped_mm(X, offsets, W, bias=None, Y=None):
    """Y[r] = X[r] W[e]^T (+ bias[e]) for the rows of every expert; others as in Y (zeros)."""
    X, W = _f64(X), _f64(W)
    Y = np.zeros((X.shape[0], W.shape[1])) if Y is None else _f64(Y).copy()
    for e in range(W.shape[0]):
        i, j = int(offsets[e]), int(offsets[e + 1])
        if j > i:
            Y[i:j] = X[i:j] @ W[e].T + (0.0 if bias is None else _f64(bias)[e])
    return Y


def grouped_mm_grad(dY, X, offsets, W):
    """(dX, dW, dbias) of grouped_mm (rows of no expert: zeros)."""
    dY, X, W = _f64(dY), _f64(X), _f64(W)
    dX, dW, db = np.zeros(X.shape), np.zeros(W.shape), np.zeros(W.shape[:2])
    for e in range(W.shape[0]):
        i, j = int(offsets[e]), int(offsets[e + 1])
        if j > i:
            dX[i:j] = dY[i:j] @ W[e]
            dW[e] = dY[i:j].T @ X[i:j]
            db[e] = dY[i:j].sum(0)
    return dX, dW, db
