"""float64 oracle of routing, sorting, dispatch / combine and 4-bit microscaled rows.

TEST INFRASTRUCTURE ONLY (see the package docstring).  Plain numpy, written from the formulas that
``include/rd_moe.h`` states, token by token and block by block.
"""
from __future__ import annotations

from typing import Optional

import numpy as np

SOFTMAX, SIGMOID = 0, 1
LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


# ---------------------------------------------------------------------------- routing
def sigmoid(x):
    x = np.asarray(x, np.float64)
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-x))


def route_keys(logits, bias, score):
    """Selection keys of one token; -inf for a masked expert."""
    l = np.asarray(logits, np.float64)
    masked = np.isnan(l) | np.isneginf(l)
    key = l if score == SOFTMAX else sigmoid(l)
    if bias is not None:
        key = key + np.asarray(bias, np.float64)
    return np.where(masked, -np.inf, key)


def route_choose(logits, bias, topk, score, groups=1, topk_groups=None):
    """Expert ids of one token, best first (-1 where none is left)."""
    key = route_keys(logits, bias, score)
    size = len(key) // groups
    topk_groups = groups if topk_groups is None else topk_groups
    if groups > 1:
        scores = []
        for g in range(groups):
            part = sorted(key[g * size:(g + 1) * size], reverse=True)
            s = part[0]
            if score == SIGMOID and size > 1 and part[1] > -np.inf:
                s = s + part[1]
            scores.append(s)
        kept = sorted((g for g in range(groups) if scores[g] > -np.inf),
                      key=lambda g: (-scores[g], g))[:topk_groups]
        for g in range(groups):
            if g not in kept:
                key[g * size:(g + 1) * size] = -np.inf
    order = sorted((e for e in range(len(key)) if key[e] > -np.inf), key=lambda e: (-key[e], e))
    return (order + [-1] * topk)[:topk]


def route_weights(logits, ids, score, renorm, scale=1.0):
    """Weights of the chosen ids of one token."""
    l = np.asarray(logits, np.float64)
    live = ~(np.isnan(l) | np.isneginf(l))
    w = np.zeros(len(ids))
    at = [(k, e) for k, e in enumerate(ids) if 0 <= e < len(l)]
    if not at:
        return w
    chosen = np.array([l[e] for _, e in at])
    if score == SOFTMAX:
        over = chosen if renorm else l[live]
        top = over.max()
        part, total = np.exp(chosen - top), np.exp(over - top).sum()
    else:
        part = sigmoid(chosen)
        total = part.sum() if renorm else 1.0
    for (k, _), p in zip(at, part):
        w[k] = scale * p / total if total > 0 else 0.0
    return w


def route_loss_grad(logits, ids, d_weights, score, renorm, scale=1.0):
    """d/dlogits of sum_k d_weights[k] * weight[k] for one token, choice held fixed."""
    l = np.asarray(logits, np.float64)
    live = ~(np.isnan(l) | np.isneginf(l))
    g = np.zeros(len(l))
    at = [(k, e) for k, e in enumerate(ids) if 0 <= e < len(l)]
    if not at:
        return g
    q = route_weights(l, ids, score, renorm)
    d = np.asarray(d_weights, np.float64)
    mean = sum(q[k] * d[k] for k, _ in at)
    if score == SOFTMAX and not renorm:
        p = np.where(live, np.exp(np.where(live, l, 0.0) - l[live].max()), 0.0)
        g = -scale * p / p.sum() * mean
        for k, e in at:
            g[e] += scale * q[k] * d[k]
    else:
        s = {e: sigmoid(l[e]) for _, e in at}
        total = sum(s.values())
        for k, e in at:
            if score == SOFTMAX:
                g[e] = scale * q[k] * (d[k] - mean)
            elif renorm:
                g[e] = scale / total * (d[k] - mean) * s[e] * (1 - s[e]) if total > 0 else 0.0
            else:
                g[e] = scale * d[k] * s[e] * (1 - s[e])
    return g


# ---------------------------------------------------------------------------- packed rows
def sort_rows(ids, experts: int, limit: Optional[int] = None, pos_prior=None):
    """(group_sizes, pos, rows); pos of tokens at or past the limit keeps pos_prior."""
    ids = np.asarray(ids)
    L = len(ids) if limit is None else max(0, min(int(limit), len(ids)))
    pos = np.full(ids.shape, -1) if pos_prior is None else np.array(pos_prior)
    row, sizes = 0, np.zeros(experts, np.int64)
    pos[:L] = -1
    for e in range(experts):
        for t, k in np.argwhere(ids[:L] == e):
            pos[t, k] = row
            row += 1
            sizes[e] += 1
    return sizes, pos, row


def combine_rows(y, pos, w):
    """(value, sum of the magnitudes of its terms) of sum_k w y[pos], float64."""
    y = np.asarray(y, np.float64)
    out = np.zeros((len(pos), y.shape[1]))
    mag = np.zeros_like(out)
    for t in range(len(pos)):
        for k, p in enumerate(pos[t]):
            if 0 <= p < len(y):
                term = (1.0 if w is None else float(w[t, k])) * y[p]
                out[t] += term
                mag[t] += np.abs(term)
    return out, mag


# ---------------------------------------------------------------------------- 4-bit rows
def mx_scale_byte(amax):
    """E8M0 byte of a block from its largest magnitude (255 where it is not finite)."""
    if not np.isfinite(amax):
        return 255
    if amax == 0:
        return 0
    return max(int(np.floor(np.log2(amax))) - 2 + 127, 0)


def mx_round(v):
    """Nearest E2M1 code (sign in bit 3) of finite values, ties to the even code, above 6 to 6."""
    a = np.abs(np.asarray(v, np.float64))
    far = np.abs(a[..., None] - LEVELS)
    best = far.min(-1, keepdims=True)
    near = far == best
    # of two equally near levels one has an even code
    even = near & (np.arange(8) % 2 == 0)
    code = np.where(even.any(-1), even.argmax(-1), near.argmax(-1))
    return (code | (np.signbit(v).astype(np.int64) << 3)).astype(np.uint8)


def mx_quantize(x):
    """Codes (one to an element) and scale bytes of rows, in blocks of 32."""
    x = np.asarray(x, np.float64)
    blocks = x.reshape(*x.shape[:-1], -1, 32)
    amax = np.abs(blocks).max(-1)
    byte = np.vectorize(mx_scale_byte, otypes=[np.int64])(np.where(np.isnan(blocks).any(-1), np.nan, amax))
    with np.errstate(invalid="ignore"):
        scaled = np.where((byte == 255)[..., None], 0.0, blocks / np.exp2(byte - 127.0)[..., None])
    return mx_round(scaled).reshape(x.shape), byte.astype(np.uint8)


def mx_values(codes, scale_bytes):
    """float64 values of codes and their blocks' scale bytes (NaN for byte 255)."""
    codes = np.asarray(codes)
    mag = LEVELS[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    s = np.where(scale_bytes == 255, np.nan, np.exp2(scale_bytes.astype(np.float64) - 127.0))
    return (mag.reshape(*scale_bytes.shape, 32) * s[..., None]).reshape(codes.shape)


def mx_pack(codes):
    """Two codes a byte, the first in the low half."""
    codes = np.asarray(codes, np.uint8)
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def mx_unpack(q):
    q = np.asarray(q, np.uint8)
    return np.stack((q & 15, q >> 4), -1).reshape(*q.shape[:-1], 2 * q.shape[-1])
