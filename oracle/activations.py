"""Activation checkpoints, the gradients made from them, and embeddings, in numpy: codes and scales bit for bit, computed
values in 64 bits from the definition."""

import numpy as np
from math import erfc

from .tensor_set import E4M3, e4m3_nearest, scale_bytes

BLOCK = 32
KINDS = ("relu", "silu", "gelu", "gelu_tanh")


def blocks(cols):
    return -(-cols // BLOCK)


def store(x):
    """(codes [rows, 32 blocks], scales [rows, blocks]) of a matrix of fp32 values."""
    x = np.asarray(x, np.float32)
    rows, cols = x.shape
    b = blocks(cols)
    y = np.zeros((rows, b * BLOCK), np.float32)
    y[:, :cols] = x
    y = y.reshape(rows, b, BLOCK)
    bad = ~np.isfinite(y).all(2)
    top = np.where(bad, 0, np.abs(np.where(np.isfinite(y), y, 0)).max(2)).astype(np.float32)
    s = scale_bytes(top.reshape(-1)).reshape(rows, b).astype(np.int64)
    with np.errstate(invalid="ignore"):
        scaled = np.ldexp(y.astype(np.float64), (127 - s)[:, :, None])
        most = np.where(s < 247, 448.0, 240.0)[:, :, None]      # 240 2^120 is the largest finite number
        scaled = np.clip(scaled, -most, most)
    code = e4m3_nearest(np.where(bad[:, :, None], 0, scaled).astype(np.float32)).reshape(rows, b, BLOCK)
    code = np.where(bad[:, :, None], 0x7F, code).astype(np.uint8).reshape(rows, b * BLOCK)
    code[:, cols:] = 0
    return code, np.where(bad, 255, s).astype(np.uint8)


def load(code, scale, cols):
    """The values of a checkpoint, in 64 bits."""
    rows, b = scale.shape
    v = E4M3[code].reshape(rows, b, BLOCK)
    v = np.where(scale[:, :, None] == 255, np.nan, np.ldexp(v, scale.astype(np.int64)[:, :, None] - 127))
    return v.reshape(rows, b * BLOCK)[:, :cols]


_erfc = np.vectorize(erfc, otypes=[np.float64])


def angle(kind, z):
    """What the exponential of an activation is taken of."""
    if kind == "gelu":
        return z * z / 2
    if kind == "gelu_tanh":
        return 2 * np.sqrt(2 / np.pi) * (z + 0.044715 * z ** 3)
    return z


def act(kind, z):
    """(act(z), act'(z), |act'(z)| with its two terms' magnitudes added) in 64 bits."""
    z = np.asarray(z, np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        if kind == "relu":
            d = np.where(z > 0, 1.0, np.where(z <= 0, 0.0, z))
            return np.where(z <= 0, 0.0, z), d, np.abs(d)
        if kind == "gelu":
            p = 0.5 * _erfc(-z / np.sqrt(2.0))
            q = z * np.exp(-z * z / 2) / np.sqrt(2 * np.pi)
        else:
            a = angle(kind, z)
            p = 1 / (1 + np.exp(-a))
            slope = 1.0 if kind == "silu" else 2 * np.sqrt(2 / np.pi) * (1 + 3 * 0.044715 * z * z)
            q = z * p / (1 + np.exp(a)) * slope
        return z * p, p + q, p + np.abs(q)


def weight_grad(dy, x):
    """(dw [n, k], bias [n]) and the sums of their summands' magnitudes."""
    dy = np.asarray(dy, np.float64)
    return (dy.T @ x, dy.sum(0)), (np.abs(dy).T @ np.abs(x), np.abs(dy).sum(0))


def lookup(table, tokens, first, scale):
    r = tokens.astype(np.int64) - first
    ok = (r >= 0) & (r < len(table))
    out = np.zeros((len(tokens), table.shape[1]), np.float64)
    out[ok] = np.asarray(table, np.float64)[r[ok]] * scale
    return out


def embedding_grad(dy, tokens, rows, first, scale):
    """(the table's gradient, its summands' magnitudes, how many summands each row has)"""
    r = tokens.astype(np.int64) - first
    ok = (r >= 0) & (r < rows)
    out, mag = np.zeros((rows, dy.shape[1])), np.zeros((rows, dy.shape[1]))
    dy = np.asarray(dy, np.float64)[ok] * scale
    np.add.at(out, r[ok], dy)
    np.add.at(mag, r[ok], np.abs(dy))
    return out, mag, np.bincount(r[ok], minlength=rows)
