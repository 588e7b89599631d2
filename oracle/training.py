"""Plain 64-bit implementations of the training operators (numpy): embedding
lookup and its gradient, layer norm, counter-based dropout and the preference
loss.  TEST INFRASTRUCTURE ONLY, like the rest of this package; each follows
the formula in ``include/oop.h`` with no thought for speed, and is pinned by
``tests/test_training_oracle.py``.
"""

from __future__ import annotations

import numpy as np

import oracle


def get_rows(table_values, ids, scale):
    """table_values: (V, M) float64; rows of ids outside [0, V) are 0."""
    y = np.zeros((len(ids), table_values.shape[1]))
    for t, i in enumerate(ids):
        if 0 <= i < len(table_values):
            y[t] = scale * table_values[i]
    return y


def table_values(raw, type_id, M):
    """float64 (V, M) of raw rows (uint8 blocks or 2- or 4-byte elements)."""
    raw = np.ascontiguousarray(raw)
    return np.stack([oracle.dequant_row(type_id, row, M) for row in raw])


def get_rows_back(dy, ids, n_rows, scale):
    """(gradient, sum of magnitudes, occurrences) in float64."""
    d, mag = np.zeros((n_rows, dy.shape[1])), np.zeros((n_rows, dy.shape[1]))
    count = np.zeros(n_rows, dtype=np.int64)
    for t, i in enumerate(ids):
        if 0 <= i < n_rows:
            d[i] += scale * dy[t]
            mag[i] += np.abs(scale * dy[t])
            count[i] += 1
    return d, mag, count


def layer_norm(x, w, b, eps):
    """(y, mean, rstd) over the last axis."""
    mean = x.mean(-1, keepdims=True)
    rstd = 1.0 / np.sqrt(((x - mean) ** 2).mean(-1, keepdims=True) + eps)
    y = (x - mean) * rstd
    if w is not None:
        y = y * w
    if b is not None:
        y = y + b
    return y, mean[..., 0], rstd[..., 0]


def layer_norm_back(dy, x, mean, rstd, w):
    xh = (x - mean[:, None]) * rstd[:, None]
    g = dy if w is None else dy * w
    dx = rstd[:, None] * (g - g.mean(1, keepdims=True) - xh * (g * xh).mean(1, keepdims=True))
    return dx, (dy * xh).sum(0), dy.sum(0)


def philox4x32_10(counter, key):
    """One call of the generator (Salmon et al., SC 2011) in Python integers."""
    c, k = [int(v) for v in counter], [int(v) for v in key]
    for _ in range(10):
        a, b = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(b >> 32) ^ c[1] ^ k[0], b & 0xFFFFFFFF, (a >> 32) ^ c[3] ^ k[1], a & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def dropout_keep(T, M, p, seed, offset):
    """Boolean (T, M): the elements that stay."""
    drop = int(np.rint(p * 65536))
    keep = np.zeros((T, M), dtype=bool)
    for t in range(T):
        for g in range((M + 7) // 8):
            r = philox4x32_10([g, t, offset & 0xFFFFFFFF, offset >> 32],
                              [seed & 0xFFFFFFFF, seed >> 32])
            for j in range(min(8, M - 8 * g)):
                keep[t, 8 * g + j] = ((r[j // 2] >> (16 * (j % 2))) & 0xFFFF) >= drop
    return keep


def dropout(x, p, seed, offset):
    drop = int(np.rint(p * 65536))
    keep = dropout_keep(x.shape[0], x.shape[1], p, seed, offset)
    scale = 65536.0 / (65536 - drop) if drop < 65536 else 0.0
    return np.where(keep, np.where(keep, x, 0.0) * scale, 0.0)


def _log_sum(x):
    top = x.max()
    return top if np.isinf(top) else top + np.log(np.exp(x - top).sum())


def _sequence_of(seq, t):
    for s in range(len(seq) - 1):
        if seq[s] <= t < seq[s + 1]:
            return s
    return -1


def preference_loss(x, labels, seq, ref, beta, e):
    """(loss, losses, ratios, logps, lse)."""
    T, P = len(labels), (len(seq) - 1) // 2
    lse, logps, ratios = np.zeros(T), np.zeros(T), np.zeros(2 * P)
    for t in range(T):
        if labels[t] < 0 or labels[t] >= x.shape[1]:
            continue
        lse[t] = _log_sum(x[t])
        logps[t] = x[t, labels[t]] - lse[t]
        s = _sequence_of(seq, t)
        if s >= 0:
            ratios[s] += logps[t] - (ref[t] if ref is not None else 0.0)
    m = beta * (ratios[:P] - ratios[P:])
    losses = (1 - e) * np.logaddexp(0.0, -m) + e * np.logaddexp(0.0, m)
    return (losses.mean() if P else 0.0), losses, ratios, logps, lse


def preference_loss_back(x, labels, seq, lse, ratios, beta, e, dloss=1.0):
    """(gradient, row coefficients)."""
    T, P = len(labels), (len(seq) - 1) // 2
    d, coef = np.zeros(x.shape), np.zeros(T)
    for t in range(T):
        s = _sequence_of(seq, t)
        if labels[t] < 0 or labels[t] >= x.shape[1] or s < 0:
            continue
        m = beta * (ratios[s % P] - ratios[P + s % P])
        c = dloss * beta / P * (e / (1 + np.exp(-m)) - (1 - e) / (1 + np.exp(m)))
        coef[t] = c if s < P else -c
        d[t] = -coef[t] * np.exp(x[t] - lse[t])
        d[t, labels[t]] += coef[t]
    return d, coef
