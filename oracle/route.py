"""The MoE router, its balance loss, their gradient, and the row layout of the
choices, in float64 and token by token.

TEST INFRASTRUCTURE ONLY (see the package docstring).

s = softmax(z) or sigmoid(z), p = s / sum(s); the k experts of largest z, or
of largest s + bias, ties to the lower index; -inf and NaN are not eligible.
w_j = scale * s_j / (sum of the chosen s, or 1).  Loss = alpha / S * sum over
the sequences of sum_i f_i P_i, f_i = E n_i / (k T_s), P_i = mean of p_i over
the T_s tokens that have an eligible expert.
"""
from __future__ import annotations

import numpy as np


def scores(z, score: int):
    """s [E] (0 where not eligible) and the eligible experts, for one token."""
    ok = ~np.isnan(z) & (z > -np.inf)
    s = np.zeros(len(z))
    if ok.any():
        if score == 0:
            e = np.exp(z[ok] - z[ok].max())
            s[ok] = e / e.sum()
        else:
            with np.errstate(over="ignore"):
                s[ok] = 1 / (1 + np.exp(-z[ok]))
    return s, ok


def choose(key, ok, k: int):
    """Indices of the k largest keys among ok, descending, ties to the lower index; -1 where there is none."""
    order = sorted((e for e in range(len(key)) if ok[e]), key=lambda e: (-key[e], e))
    return np.array((order + [-1] * k)[:k])


def route(z, k, score=0, bias=None, valid=None, seq=None, normalize=True, scale=1.0, alpha=0.0, idx=None):
    """(idx, w, counts, tokens, loss).  `idx` gives the choice instead of making it."""
    z = np.asarray(z, np.float64)
    T, E = z.shape
    seq = np.array([0, T]) if seq is None else np.asarray(seq)
    S = len(seq) - 1
    out_idx, w = np.full((T, k), -1, np.int64), np.zeros((T, k))
    p = np.zeros((T, E))
    live = np.zeros(T, bool)
    for t in range(T):
        if valid is not None and not valid[t]:
            continue
        s, ok = scores(z[t], score)
        live[t] = ok.any()
        p[t] = s / (s.sum() + 1e-20)
        out_idx[t] = idx[t] if idx is not None else choose(s + bias if bias is not None else z[t], ok, k)
        sel = out_idx[t] >= 0
        ws = np.where(sel, s[out_idx[t]], 0)
        w[t] = scale * ws / ((ws.sum() + 1e-20) if normalize else 1)
    counts, tokens, loss = np.zeros((S, E), np.int64), np.zeros(S, np.int64), 0.0
    for q in range(S):
        t = np.arange(seq[q], seq[q + 1])
        c = out_idx[t].reshape(-1)
        counts[q] = np.bincount(c[c >= 0], minlength=E)
        tokens[q] = live[t].sum()
        if tokens[q]:
            loss += (E * counts[q] / (k * tokens[q]) * p[t].sum(0) / tokens[q]).sum()
    return out_idx, w, counts, tokens, alpha / S * loss


def backward(z, idx, dw, dloss, score=0, valid=None, seq=None, normalize=True, scale=1.0, alpha=0.0):
    """d logits, by the Jacobian of each token: explicit matrices, no closed forms shared with the kernel."""
    z = np.asarray(z, np.float64)
    T, E = z.shape
    k = idx.shape[1]
    seq = np.array([0, T]) if seq is None else np.asarray(seq)
    S = len(seq) - 1
    _, _, counts, tokens, _ = route(z, k, score, None, valid, seq, normalize, scale, alpha, idx)
    dz = np.zeros((T, E))
    for q in range(S):
        for t in range(seq[q], seq[q + 1]):
            if valid is not None and not valid[t]:
                continue
            s, ok = scores(z[t], score)
            if not ok.any():
                continue
            n = tokens[q]
            dp = dloss * alpha / S * E * counts[q] / (k * n) / n
            total = s.sum()
            dp_ds = np.eye(E) / total - np.outer(s, np.ones(E)) / total ** 2        # p = s / sum(s)
            ds = dp_ds.T @ dp
            sel = [j for j in range(k) if idx[t, j] >= 0]
            chosen = sum(s[idx[t, j]] for j in sel)
            for j in sel:
                for i in sel if normalize else [j]:
                    d = scale * ((i == j) / chosen - s[idx[t, j]] / chosen ** 2) if normalize else scale
                    ds[idx[t, i]] += dw[t, j] * d
            ds_dz = np.diag(s) - np.outer(s, s) if score == 0 else np.diag(s * (1 - s))
            dz[t] = np.where(ok, ds_dz.T @ ds, 0)
    return dz


def layout(idx, E: int, rows: int):
    """(offsets, row_token, row_of): the choices expert by expert, in token order, segments padded to 128."""
    T, k = idx.shape
    offsets, row_token, row_of = np.zeros(E + 1, np.int64), np.full(rows, -1), np.full((T, k), -1)
    at = 0
    for e in range(E):
        offsets[e] = at
        for t in range(T):
            for j in range(k):
                if idx[t, j] == e:
                    row_token[at], row_of[t, j] = t, at
                    at += 1
        at = -(-at // 128) * 128
    offsets[E] = at
    return offsets, row_token, row_of
