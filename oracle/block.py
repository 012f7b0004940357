"""The operators between a block's products in float64 numpy (TEST
INFRASTRUCTURE ONLY), written as plain loops from their definitions.

``append`` places rows in a paged cache after per-head norm and rotation,
``attend`` runs one softmax per token and query head over the keys it sees,
``residual_norm`` the residual step.  Each returns the float64 values and,
where a tolerance needs it, the sums of absolute terms a rounding error scales
with.  Pinned in tests/test_block_cpu.py by hand-worked cases.
"""
from __future__ import annotations

import math

import numpy as np


def rms_norm(x, weight, eps, offset=0.0):
    x = np.asarray(x, dtype=np.float64)
    r = np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
    return x / r * (np.asarray(weight, dtype=np.float64) + offset)


def rotate(x, position, inv_freq, interleaved=False, amplitude=1.0):
    """One head row: the first 2 * len(inv_freq) elements turned in pairs."""
    x = np.array(x, dtype=np.float64)
    half = len(inv_freq)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        angle = float(position) * float(inv_freq[i])
        c, s = amplitude * math.cos(angle), amplitude * math.sin(angle)
        x[a], x[b] = x[a] * c - x[b] * s, x[b] * c + x[a] * s
    return x


def append(k_cache, v_cache, q, k, v, positions, slots, inv_freq=(), interleaved=False,
           amplitude=1.0, q_norm=None, k_norm=None, eps=1e-6, offset=0.0):
    """(q_out [n, hq, dim], k_cache, v_cache), float64: caches [pages, heads,
    page, dim] copied and written at slots; a slot outside them writes nothing."""
    kc, vc = np.array(k_cache, dtype=np.float64), np.array(v_cache, dtype=np.float64)
    pages, heads, page, dim = kc.shape
    n = len(slots)

    def made(row, t, weight):
        row = np.asarray(row, dtype=np.float64)
        if weight is not None:
            row = rms_norm(row, weight, eps, offset)
        if len(inv_freq):
            row = rotate(row, positions[t], inv_freq, interleaved, amplitude)
        return row

    q = np.asarray(q).reshape(n, -1, dim)
    out = np.empty(q.shape, dtype=np.float64)
    k, v = np.asarray(k).reshape(n, heads, dim), np.asarray(v).reshape(n, heads, dim)
    for t in range(n):
        for h in range(q.shape[1]):
            out[t, h] = made(q[t, h], t, q_norm)
        if 0 <= slots[t] < pages * page:
            at, off = divmod(int(slots[t]), page)
            for h in range(heads):
                kc[at, h, off] = made(k[t, h], t, k_norm)
                vc[at, h, off] = v[t, h]
    return out, kc, vc


def sees(p, j, window=0, sinks=0):
    """Whether the token at position p sees key j."""
    if j > p:
        return False
    return window == 0 or j > p - window or j < sinks


def attend(k_cache, v_cache, q, q_start, kv_len, table, window=0, sinks=0, scale=1.0):
    """(y, absolute, score): y [n, hq, dim] float64, NaN where no conversation
    holds the token; absolute = sum_j w_j |v_j|; score [n, hq] the largest
    scale * sum_d |q_d k_jd| over the keys the row sees (0 if none)."""
    kc, vc = np.asarray(k_cache, dtype=np.float64), np.asarray(v_cache, dtype=np.float64)
    pages, heads, page, dim = kc.shape
    q = np.asarray(q, dtype=np.float64)
    n, hq, _ = q.shape
    y = np.full((n, hq, dim), np.nan)
    absolute, score = np.zeros((n, hq, dim)), np.zeros((n, hq))
    for s in range(len(kv_len)):
        new = q_start[s + 1] - q_start[s]
        for i in range(new):
            t, p = q_start[s] + i, kv_len[s] - new + i
            js = [j for j in range(p + 1) if sees(p, j, window, sinks)]
            if not js:
                y[t] = 0.0
                continue
            where = [int(table[s][j // page]) if j // page < len(table[s]) else -1 for j in js]
            if any(w < 0 or w >= pages for w in where):
                continue                                   # NaN
            offs = [j % page for j in js]
            for h in range(hq):
                c = h // (hq // heads)
                kk, vv = kc[where, c, offs], vc[where, c, offs]
                z = scale * (kk @ q[t, h])
                w = np.exp(z - z.max())
                w /= w.sum()
                y[t, h] = w @ vv
                absolute[t, h] = w @ np.abs(vv)
                score[t, h] = scale * (np.abs(kk) @ np.abs(q[t, h])).max()
    return y, absolute, score


def residual_norm(h, b=None, pre=None, post=None, gate=None, alpha=1.0, eps=1e-6, offset=0.0):
    """(h_out, y), float64; y None without pre."""
    h = np.asarray(h, dtype=np.float64)
    if b is not None:
        b = np.asarray(b, dtype=np.float64)
        if post is not None:
            b = rms_norm(b, post, eps, offset)
        if gate is not None:
            b = b * np.asarray(gate, dtype=np.float64)
        h = h + alpha * b
    return h, None if pre is None else rms_norm(h, pre, eps, offset)
