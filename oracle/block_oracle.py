"""fp64 oracle of the feed-forward block's operations: layer norm and its
vector-Jacobian product, the gated projection and its own, and activations
kept in 8 bits.  numpy only; written from the formulas of include/mlp_ops.h,
without the library's code.
"""
from __future__ import annotations

import numpy as np

ACT_NONE, ACT_RELU, ACT_GELU_TANH, ACT_SILU = 0, 1, 2, 3
Q8_BLOCK = 32


# ---- layer norm ----------------------------------------------------------
def layer_norm(x, gamma=None, beta=None, eps=1e-5):
    """(y, mean, rstd) of each row of x [M, D]."""
    mean = x.mean(axis=1)
    d = x - mean[:, None]
    rstd = 1.0 / np.sqrt((d * d).mean(axis=1) + eps)
    y = d * rstd[:, None]
    if gamma is not None:
        y = y * gamma
    if beta is not None:
        y = y + beta
    return y, mean, rstd


def layer_norm_vjp(dy, x, mean, rstd, gamma=None):
    """(dx, dgamma, dbeta) for the statistics given."""
    xh = (x - mean[:, None]) * rstd[:, None]
    w = dy if gamma is None else dy * gamma
    dx = rstd[:, None] * (w - w.mean(axis=1, keepdims=True) - xh * (w * xh).mean(axis=1, keepdims=True))
    return dx, (dy * xh).sum(axis=0), dy.sum(axis=0)


# ---- the gated projection -------------------------------------------------
def _sigmoid(t):
    e = np.exp(-np.abs(t))
    return np.where(t >= 0, 1.0, e) / (1.0 + e)


def act(g, kind):
    if kind == ACT_NONE:
        return g
    if kind == ACT_RELU:
        return np.maximum(g, 0.0)
    if kind == ACT_SILU:
        return g * _sigmoid(g)
    # 0.5 g (1 + tanh(c)) = g / (1 + e^{-2c}); 1 + tanh(c) itself would cancel far down the left tail
    return g * _sigmoid(2.0 * np.sqrt(2.0 / np.pi) * (g + 0.044715 * g ** 3))


def act_grad(g, kind):
    if kind == ACT_NONE:
        return np.ones_like(g)
    if kind == ACT_RELU:
        return (g > 0).astype(np.float64)
    if kind == ACT_SILU:
        return _sigmoid(g) + g * _sigmoid(g) * _sigmoid(-g)
    c = 2.0 * np.sqrt(2.0 / np.pi)
    t = c * (g + 0.044715 * g ** 3)
    return _sigmoid(t) + g * _sigmoid(t) * _sigmoid(-t) * c * (1.0 + 3 * 0.044715 * g * g)


def gated_linear(x, w, b, kind):
    """(h, s): s = x w^T + b [M, 2F], h = act(s[:, :F]) * s[:, F:]."""
    s = x @ w.T
    if b is not None:
        s = s + b
    F = w.shape[0] // 2
    return act(s[:, :F], kind) * s[:, F:], s


def gated_vjp(dh, s, kind):
    """(ds, h) from the gradient dh of h and the pre-activations s."""
    F = s.shape[1] // 2
    g, u = s[:, :F], s[:, F:]
    a = act(g, kind)
    return np.concatenate([dh * u * act_grad(g, kind), dh * a], axis=1), a * u


# ---- 8-bit checkpoints ------------------------------------------------------
def _e4m3_table():
    """Values of the codes 0 .. 126 (the positive finite ones), ascending."""
    return np.array([(c & 7) / 512.0 if c < 8 else (1 + (c & 7) / 8.0) * 2.0 ** ((c >> 3) - 7) for c in range(127)])


def q8_encode(x):
    """(codes, scale bytes) of x [rows, cols] (fp64 holding fp32 or bf16 values)."""
    rows, cols = x.shape
    table = _e4m3_table()
    nb = -(-cols // Q8_BLOCK)
    q = np.zeros((rows, cols), np.uint8)
    e = np.zeros((rows, nb), np.uint8)
    for b in range(nb):
        v = x[:, b * Q8_BLOCK:(b + 1) * Q8_BLOCK]
        fin = np.isfinite(v)
        top = np.where(fin, np.abs(v), 0.0).max(axis=1)
        k = np.full(rows, -120)
        while np.any(top > 448.0 * 2.0 ** k.astype(np.float64)):
            k += top > 448.0 * 2.0 ** k.astype(np.float64)
        e[:, b] = k + 127
        s = np.where(fin, np.abs(v), 0.0) * 2.0 ** -k.astype(np.float64)[:, None]
        hi = np.searchsorted(table, s)                     # first code whose value >= s
        hi = np.minimum(hi, 126)
        lo = np.maximum(hi - 1, 0)
        dl, dh = s - table[lo], table[hi] - s
        code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
        code = np.where(s == table[hi], hi, code)
        code = np.where(fin, code, 127) | (np.signbit(v).astype(np.int64) << 7)
        q[:, b * Q8_BLOCK:(b + 1) * Q8_BLOCK] = code
    return q, e


def q8_decode(q, e):
    """The values that codes and scale bytes stand for (fp64); scale byte 255 is NaN."""
    table = np.append(_e4m3_table(), np.nan)
    sign = np.where(q >> 7, -1.0, 1.0)
    k = np.repeat(e.astype(np.int64) - 127, Q8_BLOCK, axis=1)[:, :q.shape[1]]
    return sign * table[q & 127] * np.where(k == 128, np.nan, 2.0 ** k.astype(np.float64))
