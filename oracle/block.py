"""Norm, epilogue and experts of a transformer block in 64 bits."""

import math

import numpy as np

ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")
_erf = np.vectorize(math.erf, otypes=[np.float64])


def rms_norm(h, weight, eps):
    """(v, rstd): v = h * rstd * weight, rstd = 1 / sqrt(mean(h^2) + eps)."""
    h = np.asarray(h, np.float64)
    rstd = 1.0 / np.sqrt((h * h).mean(1) + eps)
    return h * rstd[:, None] * np.asarray(weight, np.float64), rstd


def rms_norm_bwd(dy, h, weight, eps, dh=None):
    """(dx, dw): gradients of sum(dy * v) (+ sum(dh * h)) by h and by weight."""
    h, dy, w = (np.asarray(a, np.float64) for a in (h, dy, weight))
    rstd = 1.0 / np.sqrt((h * h).mean(1, keepdims=True) + eps)
    n = h * rstd
    dx = rstd * (dy * w - n * (dy * w * n).mean(1, keepdims=True))
    return dx + (0.0 if dh is None else np.asarray(dh, np.float64)), (dy * n).sum(0)


def act(z, kind):
    z = np.asarray(z, np.float64)
    if kind == "relu":
        return np.maximum(z, 0.0)
    if kind == "silu":
        return z / (1.0 + np.exp(-z))
    if kind == "gelu":
        return 0.5 * z * (1.0 + _erf(z / math.sqrt(2.0)))
    if kind == "gelu_tanh":
        return 0.5 * z * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z**3)))
    return z


def act_slope(z, kind):
    z = np.asarray(z, np.float64)
    if kind == "relu":
        return (z > 0).astype(np.float64)
    if kind == "silu":
        s = 1.0 / (1.0 + np.exp(-z))
        return s + z * s * (1.0 - s)
    if kind == "gelu":
        return 0.5 * (1.0 + _erf(z / math.sqrt(2.0))) + z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if kind == "gelu_tanh":
        a = math.sqrt(2.0 / math.pi)
        t = np.tanh(a * (z + 0.044715 * z**3))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * a * (1.0 + 3 * 0.044715 * z * z)
    return np.ones_like(z)


def experts(x, idx, w, w1, w2, first_expert=0):
    """y[t] = sum over choices j of w[t, j] * down(silu(gate x) * up x) of expert idx[t, j], those of
    [first_expert, first_expert + G): w1 [G, 2 I, H] (gate rows first), w2 [G, H, I], all values."""
    x = np.asarray(x, np.float64)
    G, two_i, _ = w1.shape
    inner = two_i // 2
    y = np.zeros_like(x)
    for t in range(x.shape[0]):
        for j, e in enumerate(np.asarray(idx)[t] - first_expert):
            if 0 <= e < G:
                g = w1[e] @ x[t]
                y[t] += w[t, j] * (w2[e] @ (act(g[:inner], "silu") * g[inner:]))
    return y
