"""Definitions in fp64 of the operators of a distillation step: RMS norm with
the residual's addition (and its 8-bit output), its gradient, the product of
8-bit integers with scales, and the loss on a teacher's top logits with its
gradient.  Test infrastructure: plain numpy, no code shared with the CUDA path.
"""
from __future__ import annotations

import numpy as np


def rmsnorm(x, residual, gamma, eps):
    """(h, rstd, y): h = x + residual, rstd = 1/sqrt(mean(h²) + eps), y = h·rstd·γ per row."""
    h = np.asarray(x, np.float64)
    if residual is not None:
        h = h + np.asarray(residual, np.float64)
    rstd = 1.0 / np.sqrt(np.mean(h * h, axis=1) + eps)
    y = h * rstd[:, None]
    if gamma is not None:
        y = y * np.asarray(gamma, np.float64)
    return h, rstd, y


def rmsnorm_q8_scale(y):
    """The scale of each row's 8-bit output: max|y| / 127."""
    return np.max(np.abs(y), axis=1) / 127.0


def rmsnorm_grad(dy, h, rstd, gamma, dh):
    """(dx, dγ) with n = h·rstd, c = mean(dy·γ·n): dx = rstd·(dy·γ − n·c) + dh, dγ = Σ_rows dy·n."""
    dy, n = np.asarray(dy, np.float64), np.asarray(h, np.float64) * np.asarray(rstd, np.float64)[:, None]
    dn = dy if gamma is None else dy * np.asarray(gamma, np.float64)
    c = np.mean(dn * n, axis=1, keepdims=True)
    dx = np.asarray(rstd, np.float64)[:, None] * (dn - n * c)
    if dh is not None:
        dx = dx + np.asarray(dh, np.float64)
    return dx, np.sum(dy * n, axis=0)


def q8_matmul(a, a_scale, w, w_scale):
    """(Σ_k a[m, k]·w[n, k])·a_scale[m]·w_scale[n]; the integer sum is exact (below 2^53 in fp64)."""
    acc = np.asarray(a, np.float64) @ np.asarray(w, np.float64).T
    return acc * np.asarray(a_scale, np.float64)[:, None] * np.asarray(w_scale, np.float64)


def distill_topk(logits, index, teacher, temperature, dloss=None):
    """(loss, lse, dlogits) per token, one token at a time:
    p = softmax(teacher/τ) over the entries whose index lies in the vocabulary, q = softmax(z/τ),
    loss = τ² Σ p_j (ln p_j − ln q[index_j]), dz = dloss·τ·(q − p scattered); a token without entries (or with
    −infinity in all of them) has loss and gradient 0, a token of dloss 0 gradient 0."""
    T, V = logits.shape
    loss, lse, dz = np.zeros(T), np.zeros(T), np.zeros((T, V))
    for t in range(T):
        z = np.asarray(logits[t], np.float64) / temperature
        m = np.max(z)
        lse[t] = m + np.log(np.sum(np.exp(z - m)))
        at = np.asarray(index[t], np.int64)
        ok = (at >= 0) & (at < V)
        e = np.asarray(teacher[t], np.float64)[ok] / temperature
        at = at[ok]
        if e.size == 0 or np.all(e == -np.inf):
            continue
        log_p = e - (np.max(e) + np.log(np.sum(np.exp(e - np.max(e)))))
        p = np.exp(log_p)
        on = p > 0
        loss[t] = temperature ** 2 * np.sum(p[on] * (log_p[on] - (z[at[on]] - lse[t])))
        g = (1.0 if dloss is None else float(dloss[t])) * temperature
        if g != 0:
            row = g * np.exp(z - lse[t])
            np.subtract.at(row, at, g * p)
            dz[t] = row
    return loss, lse, dz
