"""fp64 reference of the operators that bring tokens to their experts and back, of
the int8 products and of dropout. Test infrastructure: plain NumPy, written from
the definitions."""
from __future__ import annotations

import numpy as np


def sort(ids, experts):
    """ids [T, k] -> (rows [T, k], choices [T * k], counts [experts]), int32."""
    flat = np.asarray(ids, np.int64).ravel()
    kept = (flat >= 0) & (flat < experts)
    key = np.where(kept, flat, experts)
    choices = np.lexsort((np.arange(key.size), key)).astype(np.int32)
    place = np.empty(key.size, np.int64)
    place[choices] = np.arange(key.size)
    rows = np.where(kept, place, -1 - place).astype(np.int32).reshape(np.shape(ids))
    return rows, choices, np.bincount(key, minlength=experts + 1)[:experts].astype(np.int32)


def dispatch(x, rows, expert_rows, out=None):
    """[expert_rows, C]; rows that no place names are those of out (or NaN)."""
    x, rows = np.asarray(x, np.float64), np.asarray(rows)
    y = np.full((expert_rows, x.shape[1]), np.nan) if out is None else np.array(out, np.float64)
    for t in range(rows.shape[0]):
        for r in rows[t]:
            if r >= 0 and r < expert_rows:
                y[r] = x[t]
            elif r < 0 and ~r < expert_rows:
                y[~r] = 0
    return y


def combine(y, rows, weights=None):
    """(out [T, C], sum of magnitudes [T, C])."""
    y, rows = np.asarray(y, np.float64), np.asarray(rows)
    T, k = rows.shape
    w = np.ones((T, k)) if weights is None else np.asarray(weights, np.float64)
    out, size = np.zeros((T, y.shape[1])), np.zeros((T, y.shape[1]))
    for t in range(T):
        for j in range(k):
            if 0 <= rows[t, j] < y.shape[0]:
                v = w[t, j] * y[rows[t, j]]
                out[t] += v
                size[t] += np.abs(v)
    return out, size


def combine_bwd(dout, y, rows, weights, out=None):
    """(dy, dweights, sum of the magnitudes of a weight's products)."""
    dout, y, rows = np.asarray(dout, np.float64), np.asarray(y, np.float64), np.asarray(rows)
    w = np.asarray(weights, np.float64)
    T, k = rows.shape
    dy = np.full(y.shape, np.nan) if out is None else np.array(out, np.float64)
    dw, size = np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            r = rows[t, j]
            if 0 <= r < y.shape[0]:
                dy[r] = w[t, j] * dout[t]
                dw[t, j] = (dout[t] * y[r]).sum()
                size[t, j] = np.abs(dout[t] * y[r]).sum()
            elif r < 0 and ~r < y.shape[0]:
                dy[~r] = 0
    return dy, dw, size


def quantize_int8(x):
    """x [R, K] (bf16 values in float64) -> (codes int8, scales float32)."""
    x = np.asarray(x, np.float64)
    amax = np.abs(x).max(1)            # NaN where a row holds one
    plain = np.isfinite(amax) & (amax > 0)
    q = np.zeros(x.shape, np.int8)
    q[plain] = np.rint(127 * x[plain] / amax[plain, None])
    return q, amax.astype(np.float32) / np.float32(127)


def grouped_int8(a_q, a_s, w_q, w_s, splits):
    """a_q [M, K], w_q [G, N, K], a_s [M], w_s [G, N] -> [M, N]."""
    out = np.zeros((a_q.shape[0], w_q.shape[1]))
    at = 0
    for g, m in enumerate(splits):
        # whole numbers below 2^53: exact
        acc = np.asarray(a_q[at:at + m], np.float64) @ np.asarray(w_q[g], np.float64).T
        out[at:at + m] = acc * np.asarray(a_s[at:at + m], np.float64)[:, None] * np.asarray(w_s[g], np.float64)
        at += m
    return out


def philox4x32(counter, key, rounds=10):
    """counter [..., 4], key [2] of 32-bit values -> [..., 4] (Salmon, Moraes,
    Dror, Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011)."""
    c = [np.asarray(counter)[..., i].astype(np.uint64) for i in range(4)]
    k0, k1 = (int(v) for v in key)
    low, sh = np.uint64(0xFFFFFFFF), np.uint64(32)
    for _ in range(rounds):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> sh) ^ c[1] ^ np.uint64(k0), b & low, (a >> sh) ^ c[3] ^ np.uint64(k1), a & low]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return np.stack(c, -1)


def dropout_numbers(rows, cols, seed, step, call):
    """The 16-bit number of every element."""
    groups = -(-cols // 8)
    b = np.arange(rows * groups, dtype=np.uint64)
    counter = np.stack([b & np.uint64(0xFFFFFFFF), b >> np.uint64(32), np.full_like(b, call),
                        np.full_like(b, step % 2 ** 32)], -1)
    seed %= 2 ** 64
    w = philox4x32(counter, (seed % 2 ** 32, seed // 2 ** 32))
    halves = np.stack([w & np.uint64(0xFFFF), w >> np.uint64(16)], -1)      # [blocks, 4, 2]
    return halves.reshape(rows, groups * 8)[:, :cols].astype(np.int64)


def dropout(x, p, seed, step, call, residual=None):
    """(out, kept)."""
    x = np.asarray(x, np.float64)
    limit = int(np.rint(np.float64(np.float32(p)) * 65536))
    kept = dropout_numbers(*x.shape, seed, step, call) >= limit
    scale = 65536 / (65536 - limit) if limit < 65536 else 0.0
    out = np.where(kept, np.where(kept, x, 0) * scale, 0.0)
    return (out if residual is None else out + np.asarray(residual, np.float64)), kept
