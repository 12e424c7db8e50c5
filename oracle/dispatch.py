"""Gradients of the rows sorted by expert and of the weighted sum back, in float64.

Xp[r] = X[t] and Y[t] = sum_j w[t, j] Yp[r], with r = assign_row[t k + j]; rows
outside [0, n_rows) are picks that were left out: they add nothing and get nothing."""
from __future__ import annotations

import numpy as np


def _rows(assign_row, n_rows):
    a = np.asarray(assign_row, dtype=np.int64).reshape(-1)
    n = a.size if n_rows is None else min(int(n_rows), a.size)
    return a, (a >= 0) & (a < n)


def combine_backward(dY, Yp, assign_row, w, n_rows=None):
    """-> (dYp [M, H] with NaN in rows that nothing names, dw [T, k])."""
    dY, Yp, w = (np.asarray(v, dtype=np.float64) for v in (dY, Yp, w))
    T, k = w.shape
    a, live = _rows(assign_row, n_rows)
    t = np.arange(T * k) // k
    dYp = np.full((T * k, dY.shape[1]), np.nan)
    dYp[a[live]] = w.reshape(-1)[live, None] * dY[t[live]]
    dw = np.zeros(T * k)
    dw[live] = (Yp[a[live]] * dY[t[live]]).sum(axis=1)
    return dYp, dw.reshape(T, k)


def permute_backward(dXp, assign_row, k, add=None, n_rows=None):
    """-> dX [T, H]."""
    dXp = np.asarray(dXp, dtype=np.float64)
    a, live = _rows(assign_row, n_rows)
    dX = np.zeros((a.size // k, dXp.shape[1])) if add is None else np.array(add, dtype=np.float64)
    np.add.at(dX, (np.arange(a.size) // k)[live], dXp[a[live]])
    return dX
