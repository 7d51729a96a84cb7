"""float64 oracle of layer norm, products with bias / activation / residual, and counter-based dropout.

TEST INFRASTRUCTURE ONLY (see the package docstring).  Plain numpy, written from the formulas that
``include/rd_block.h`` states.
"""
from __future__ import annotations

import math

import numpy as np

from .ragged import group_bounds

NONE, RELU, GELU, GELU_TANH, SILU = range(5)
ACTS = (NONE, RELU, GELU, GELU_TANH, SILU)


# ---------------------------------------------------------------------------- layer norm
def layer_norm(x, weight=None, bias=None, eps=1e-5):
    """(out, mean, rstd) of rows x."""
    x = np.asarray(x, np.float64)
    mean = x.mean(1)
    rstd = 1.0 / np.sqrt(((x - mean[:, None]) ** 2).mean(1) + eps)
    y = (x - mean[:, None]) * rstd[:, None]
    out = y * (1.0 if weight is None else weight) + (0.0 if bias is None else bias)
    return out, mean, rstd


def layer_norm_bwd(d_out, x, weight, mean, rstd):
    """(d_x, d_weight, d_bias) with the given statistics."""
    r = np.asarray(rstd, np.float64)[:, None]
    y = (np.asarray(x, np.float64) - np.asarray(mean, np.float64)[:, None]) * r
    d = np.asarray(d_out, np.float64)
    g = d if weight is None else d * weight
    h = y.shape[1]
    d_x = r * (g - g.sum(1, keepdims=True) / h - y * (g * y).sum(1, keepdims=True) / h)
    return d_x, (d * y).sum(0), d.sum(0)


# ---------------------------------------------------------------------------- activations
_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def normal_cdf(z):
    return 0.5 * _erfc(-np.asarray(z, np.float64) / math.sqrt(2.0)) if np.size(z) else np.zeros(np.shape(z))


def logistic(z):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-np.asarray(z, np.float64)))


_A, _C = 2.0 * math.sqrt(2.0 / math.pi), 0.044715


def act(z, kind):
    z = np.asarray(z, np.float64)
    if kind == RELU:
        return np.maximum(z, 0.0)
    if kind == GELU:
        return z * normal_cdf(z)
    if kind == GELU_TANH:
        return z * logistic(_A * (z + _C * z ** 3))
    if kind == SILU:
        return z * logistic(z)
    return z


def slope_terms(z, kind):
    """(s, b): the derivative of the activation is s + b."""
    z = np.asarray(z, np.float64)
    if kind == RELU:
        return (z > 0).astype(np.float64), np.zeros_like(z)
    if kind == GELU:
        return normal_cdf(z), z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if kind == GELU_TANH:
        s = logistic(_A * (z + _C * z ** 3))
        return s, z * s * (1 - s) * _A * (1 + 3 * _C * z * z)
    if kind == SILU:
        s = logistic(z)
        return s, z * s * (1 - s)
    return np.ones_like(z), np.zeros_like(z)


def act_slope(z, kind):
    s, b = slope_terms(z, kind)
    return s + b


# ---------------------------------------------------------------------------- products
def linear(x, w, bias=None, residual=None, kind=NONE, sizes=None, offset=0, limit=None):
    """(out, z) over rows [0, m): zero outside the local groups and past the limit.

    w [k, n] without sizes, else [g_local, k, n] (bias likewise)."""
    x = np.asarray(x, np.float64)
    if sizes is None:
        sizes, w, bias = [len(x)], w[None], None if bias is None else bias[None]
    b, L = group_bounds(sizes, len(x), limit)
    out, z = np.zeros((len(x), w.shape[2])), np.zeros((len(x), w.shape[2]))
    for j in range(len(w)):
        lo, hi = b[offset + j], b[offset + j + 1]
        z[lo:hi] = x[lo:hi] @ w[j] + (0.0 if bias is None else bias[j])
        out[lo:hi] = act(z[lo:hi], kind) + (0.0 if residual is None else residual[lo:hi])
    return out, z


def linear_act_bwd(d_out, pre, kind, sizes=None, offset=0, g_local=None, limit=None):
    """(d_pre, d_bias [g_local, n])."""
    d_out = np.asarray(d_out, np.float64)
    sizes = [len(d_out)] if sizes is None else sizes
    g_local = len(sizes) - offset if g_local is None else g_local
    b, L = group_bounds(sizes, len(d_out), limit)
    d_pre, d_bias = np.zeros_like(d_out), np.zeros((g_local, d_out.shape[1]))
    for j in range(g_local):
        lo, hi = b[offset + j], b[offset + j + 1]
        d = d_out[lo:hi] if kind == NONE else d_out[lo:hi] * act_slope(pre[lo:hi], kind)
        d_pre[lo:hi] = d
        d_bias[j] = d.sum(0)
    return d_pre, d_bias


# ---------------------------------------------------------------------------- dropout
def philox(counter, key):
    """The four words of one counter (four 32-bit words) and key (two), in ten rounds, with Python integers."""
    c, k = [int(v) for v in counter], [int(v) for v in key]
    for _ in range(10):
        a, b = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(b >> 32) ^ c[1] ^ k[0], b & 0xFFFFFFFF, (a >> 32) ^ c[3] ^ k[1], a & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def dropout_draws(seed, offset, first, vectors):
    """The 16-bit draws of vectors [first, first + vectors), [vectors, 8]."""
    low = np.uint64(0xFFFFFFFF)
    s32 = np.uint64(32)
    seed, offset = int(seed) % 2 ** 64, int(offset) % 2 ** 64
    v = np.arange(vectors, dtype=np.uint64) + np.uint64(first)
    c = [v & low, v >> s32, np.full_like(v, offset & 0xFFFFFFFF), np.full_like(v, offset >> 32)]
    k = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        a, b = np.uint64(0xD2511F53) * c[0], np.uint64(0xCD9E8D57) * c[2]
        c = [(b >> s32) ^ c[1] ^ np.uint64(k[0]), b & low, (a >> s32) ^ c[3] ^ np.uint64(k[1]), a & low]
        k = [(k[0] + 0x9E3779B9) % 2 ** 32, (k[1] + 0xBB67AE85) % 2 ** 32]
    words = np.stack(c, 1)
    return np.stack([(words >> np.uint64(16 * (i % 2)) & np.uint64(0xFFFF))[:, i // 2] for i in range(8)], 1).astype(np.int64)


def dropout_threshold(p):
    return int(math.floor(float(np.float32(p)) * 65536 + 0.5))


def dropout(x, seed, offset, p, residual=None):
    """(out, kept) of rows x."""
    x = np.asarray(x, np.float64)
    least = dropout_threshold(p)
    kept = dropout_draws(seed, offset, 0, x.size // 8).reshape(x.shape) >= least
    scale = 65536 / (65536 - least) if least < 65536 else 0.0
    out = np.where(kept, x * scale, 0.0)
    return (out if residual is None else out + residual), kept
