"""fp64 reference of the operators around the expert layer: layer norm and its
gradients, the norm of many gradients with clipping, and the whole expert layer
for a few tokens. Test infrastructure: plain NumPy, written from the formulas."""
from __future__ import annotations

import math

import numpy as np

CLIP_EPS = 1e-6


def layer_norm_fwd(x, weight=None, bias=None, eps=1e-5):
    """x [rows, cols] -> (y, mean, rstd)."""
    x = np.asarray(x, np.float64)
    mean = x.mean(1)
    rstd = 1.0 / np.sqrt(((x - mean[:, None]) ** 2).mean(1) + eps)
    y = (x - mean[:, None]) * rstd[:, None]
    if weight is not None:
        y = y * np.asarray(weight, np.float64)
    if bias is not None:
        y = y + np.asarray(bias, np.float64)
    return y, mean, rstd


def layer_norm_bwd(dy, x, weight, mean, rstd):
    """(dx, dweight, dbias) at the given mean and rstd."""
    dy, x = np.asarray(dy, np.float64), np.asarray(x, np.float64)
    mean, rstd = np.asarray(mean, np.float64)[:, None], np.asarray(rstd, np.float64)[:, None]
    xh = (x - mean) * rstd
    g = dy if weight is None else dy * np.asarray(weight, np.float64)
    dx = rstd * (g - g.mean(1, keepdims=True) - xh * (g * xh).mean(1, keepdims=True))
    return dx, (dy * xh).sum(0), dy.sum(0)


def grad_norm(grads, norm_type=2.0):
    """2: square root of the sum of squares; inf: largest magnitude (0 for no
    elements)."""
    flat = [np.asarray(g, np.float64).ravel() for g in grads]
    if norm_type == math.inf:
        return max((float(np.abs(f).max()) for f in flat if f.size), default=0.0)
    return math.sqrt(math.fsum(float((f * f).sum()) for f in flat))


def clip_factor(norm, max_norm):
    return min(1.0, max_norm / (norm + CLIP_EPS))


def route(logits, top_k, renormalize=True):
    """ids int32 [T, k] (-1: none) and weights [T, k]. -inf is never chosen, NaN
    ranks above all, equal logits go to the lowest index."""
    logits = np.asarray(logits, np.float64)
    T, E = logits.shape
    ids = np.full((T, top_k), -1, np.int32)
    weights = np.zeros((T, top_k))
    for t in range(T):
        row = logits[t]
        order = sorted((e for e in range(E) if row[e] != -math.inf),
                       key=lambda e: (not math.isnan(row[e]), -row[e] if not math.isnan(row[e]) else 0.0, e))
        pick = order[:top_k]
        if not pick:
            continue
        ids[t, :len(pick)] = pick
        with np.errstate(invalid="ignore"):
            p = np.exp(row - row[pick[0]])
            weights[t, :len(pick)] = p[pick] / (p[pick].sum() if renormalize else p.sum())
    return ids, weights


def moe_layer(x, logits, w13, w2, top_k, renormalize=True):
    """x [T, H], w13 [E, 2I, H], w2 [E, H, I] -> (y, ids, weights, bound).

    bound: how far an implementation may be that sums in fp32 and rounds the
    inner activation and the output to bf16. With u = 2^-24: a sum of K fp32
    products, in any order that adds at most 256 terms to one partial, is within
    256 u sum|a b|; |silu'| <= 1.1; a bf16 rounding is within 2^-8 |v|."""
    x = np.asarray(x, np.float64)
    ids, weights = route(logits, top_k, renormalize)
    T, H = x.shape
    inner = w2.shape[2]
    eps = 256 * 2.0 ** -24
    y, off = np.zeros((T, H)), np.zeros((T, H))
    for t in range(T):
        for e, p in zip(ids[t], weights[t]):
            if e < 0:
                continue
            a = w13[e] @ x[t]
            ea = eps * (np.abs(w13[e]) @ np.abs(x[t]))
            g, u = a[:inner], a[inner:]
            with np.errstate(over="ignore"):
                s = g / (1 + np.exp(-g))
            h = s * u
            eh = 1.1 * ea[:inner] * np.abs(u) + np.abs(s) * ea[inner:] + 1.1 * ea[:inner] * ea[inner:] \
                + (2.0 ** -8 + 2.0 ** -20) * np.abs(h)
            y[t] += p * (w2[e] @ h)
            off[t] += abs(p) * (np.abs(w2[e]) @ (eh + (eps + 2.0 ** -20) * np.abs(h)))
    return y, ids, weights, off + 2.0 ** -8 * (np.abs(y) + off)
