"""Plain 64-bit implementations (numpy) of the operators of a decoder layer's
training step: head norms with rotation, the gated feed-forward block and the
orthogonalised update.  TEST INFRASTRUCTURE ONLY, like the rest of this package;
each follows the formula in ``include/oop.h`` with no thought for speed, and is
pinned by ``tests/test_layer_oracle.py``.
"""

from __future__ import annotations

import math

import numpy as np


def pairs(D, n_rot, interleaved):
    """(first, second) elements of each rotated pair."""
    i = np.arange(n_rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + n_rot // 2)


def turned(n, pos, freqs, interleaved, sign=1):
    """n (T, H, D) with its pairs turned by sign * pos * freqs."""
    y = n.copy()
    if len(freqs) == 0:
        return y
    a, b = pairs(n.shape[-1], 2 * len(freqs), interleaved)
    angle = np.asarray(pos, dtype=np.float64)[:, None] * np.asarray(freqs, dtype=np.float64)[None, :]
    c, s = np.cos(angle)[:, None, :], sign * np.sin(angle)[:, None, :]
    y[..., a] = n[..., a] * c - n[..., b] * s
    y[..., b] = n[..., a] * s + n[..., b] * c
    return y


def norm_rope(x, w, pos, freqs, eps, interleaved):
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    n = x * r if w is None else x * r * w
    return turned(n, pos, freqs, interleaved)


def norm_rope_back(dy, x, w, pos, freqs, eps, interleaved):
    """(dx, dw)."""
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    dn = turned(dy, pos, freqs, interleaved, -1)
    g = dn if w is None else dn * w
    dx = r * (g - x * r * r * (g * x).mean(-1, keepdims=True))
    return dx, (dn * x * r).sum((0, 1))


def _erf(v):
    return np.vectorize(math.erf, otypes=[np.float64])(v) if np.size(v) else np.zeros(np.shape(v))


def _sigmoid(v):
    e = np.exp(-np.abs(v))
    return np.where(v >= 0, 1.0, e) / (1.0 + e)


def act(v, kind):
    if kind == "silu":
        return v * _sigmoid(v)
    if kind == "gelu_tanh":
        return 0.5 * v * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3)))
    if kind == "gelu_erf":
        return 0.5 * v * (1.0 + _erf(v / math.sqrt(2.0)))
    return np.maximum(v, 0.0)


def act_slope(v, kind):
    if kind == "silu":
        s = _sigmoid(v)
        return s + v * s * (1.0 - s)
    if kind == "gelu_tanh":
        k = math.sqrt(2.0 / math.pi)
        t = np.tanh(k * (v + 0.044715 * v ** 3))
        return 0.5 * (1.0 + t) + 0.5 * v * (1.0 - t * t) * k * (1.0 + 3 * 0.044715 * v * v)
    if kind == "gelu_erf":
        return 0.5 * (1.0 + _erf(v / math.sqrt(2.0))) + v * np.exp(-0.5 * v * v) / math.sqrt(2.0 * math.pi)
    return (v > 0).astype(np.float64)


def gated_ffn(x, wg, wu, kind):
    """(h, gate, up) of x (T, K) and weights (F, K)."""
    gate, up = x @ wg.T, x @ wu.T
    return act(gate, kind) * up, gate, up


def gated_ffn_back(dh, x, wg, wu, gate, up, kind):
    """(dx, dwg, dwu, dgate, dup)."""
    dg, du = dh * up * act_slope(gate, kind), dh * act(gate, kind)
    return dg @ wg + du @ wu, dg.T @ x, du.T @ x, dg, du


def orthogonalise(x, steps, coefs, eps, scale=1.0):
    """x (M, N); coefs: one (a, b, c) for each step."""
    X = x / (np.sqrt((x * x).sum()) + eps)
    for a, b, c in coefs[:steps]:
        A = X @ X.T
        X = a * X + (b * A + c * (A @ A)) @ X
    return scale * X
