"""The operators of a training step around the 8-bit products, in float64.

TEST INFRASTRUCTURE ONLY (see the package docstring).

  * rmsnorm: y = r * gain / sqrt(mean r^2 + eps), and its gradient
      dx = rstd t - r rstd^3 mean(t r) + dres   (t = dy gain),
      dgain = sum over rows of dy r rstd;
  * swiglu_backward: the gradient of silu(gate) * up;
  * combine_backward, dispatch_backward: the gradients of the weighted sum of
    each token's expert rows and of the copy of tokens into those rows;
  * grouped_wgrad: the products over each expert's rows.

Functions that sum return the magnitude of the sum as well, which bounds a
float32 sum's error.
"""
from __future__ import annotations

import numpy as np


def rmsnorm(r, gain, eps):
    """(y, rstd) of r [M, K]."""
    r, gain = np.asarray(r, np.float64), np.asarray(gain, np.float64)
    rstd = 1.0 / np.sqrt(np.mean(r * r, axis=1) + float(np.float32(eps)))
    return r * rstd[:, None] * gain, rstd


def rmsnorm_backward(dy, r, gain, rstd, dres=None):
    """(dx, its magnitude, dgain, its magnitude); rstd as given, a constant of the formula."""
    dy, r, gain = (np.asarray(v, np.float64) for v in (dy, r, gain))
    rstd = np.asarray(rstd, np.float64)[:, None]
    t = dy * gain
    dx = rstd * t - r * rstd ** 3 * np.mean(t * r, axis=1, keepdims=True)
    mag = np.abs(rstd * t) + np.abs(r) * rstd ** 3 * np.mean(np.abs(t * r), axis=1, keepdims=True)
    if dres is not None:
        dx = dx + np.asarray(dres, np.float64)
        mag = mag + np.abs(np.asarray(dres, np.float64))
    part = dy * r * rstd
    return dx, mag, part.sum(axis=0), np.abs(part).sum(axis=0)


def _sigmoid(x):
    e = np.exp(-np.abs(x))
    return np.where(x >= 0, 1.0, e) / (1.0 + e)


def swiglu_backward(h, dv, inter):
    """(dh [M, 2 inter], its magnitude) of h (gate | up) and dv, the gradient of silu(gate) * up."""
    h, dv = np.asarray(h, np.float64), np.asarray(dv, np.float64)
    g, u = h[:, :inter], h[:, inter:2 * inter]
    s, other = _sigmoid(g), _sigmoid(-g)
    dg = dv * u * s * (1.0 + g * other)
    mag = np.abs(dv * u) * s * (1.0 + np.abs(g) * other)
    du = dv * g * s
    return np.concatenate([dg, du], axis=1), np.concatenate([mag, np.abs(du)], axis=1)


def combine_backward(dout, y, row_of, w, rows):
    """(dy [rows, N], dw [T, k], dw's magnitude): dy[row] sums w dout over the slots that name it."""
    dout, y, w = (np.asarray(v, np.float64) for v in (dout, y, w))
    T, k = row_of.shape
    dy = np.zeros((rows, dout.shape[1]))
    dw, mag = np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            i = int(row_of[t, j])
            if 0 <= i < rows:
                dy[i] += w[t, j] * dout[t]
                dw[t, j] = np.dot(dout[t], y[i])
                mag[t, j] = np.dot(np.abs(dout[t]), np.abs(y[i]))
    return dy, dw, mag


def dispatch_backward(d, row_of, add=None):
    """(dx [T, N], its magnitude)."""
    d = np.asarray(d, np.float64)
    T, k = row_of.shape
    dx = np.zeros((T, d.shape[1])) if add is None else np.asarray(add, np.float64).copy()
    mag = np.abs(dx)
    for j in range(k):
        ok = (row_of[:, j] >= 0) & (row_of[:, j] < d.shape[0])
        term = np.where(ok[:, None], d[np.where(ok, row_of[:, j], 0)] if d.shape[0] else 0.0, 0.0)
        dx += term
        mag += np.abs(term)
    return dx, mag


def grouped_wgrad(a, b, offsets):
    """(D [G, N, K], its magnitude) of the values a [N, R] and b [K, R]."""
    a, b = np.asarray(a, np.float64), np.asarray(b, np.float64)
    G = len(offsets) - 1
    d = np.zeros((G, a.shape[0], b.shape[0]))
    mag = np.zeros_like(d)
    for g in range(G):
        lo, hi = int(offsets[g]), int(offsets[g + 1])
        d[g] = a[:, lo:hi] @ b[:, lo:hi].T
        mag[g] = np.abs(a[:, lo:hi]) @ np.abs(b[:, lo:hi]).T
    return d, mag
