"""The operators of a step of drafted tokens in float64 numpy (TEST
INFRASTRUCTURE ONLY), written as plain loops from their definitions.

``quantize`` and ``numbers`` are the 8-bit cache's two directions, ``rows`` the
lookup in a dequantized table, ``verify`` the acceptance of drafts and the
draw that follows.  Pinned in tests/test_step_cpu.py by hand-worked cases and,
for ``verify``, by the distribution it has to reproduce.
"""
from __future__ import annotations

import numpy as np


def quantize(x):
    """(codes int8, scale float32) of rows of float32 x, in float32 arithmetic."""
    x = np.asarray(x, dtype=np.float32)
    codes = np.zeros(x.shape, np.int8)
    scale = np.zeros(x.shape[:-1], np.float32)
    for i in np.ndindex(scale.shape):
        if not np.isfinite(x[i]).all():
            scale[i] = np.nan
            continue
        s = np.abs(x[i]).max() / np.float32(127)
        if s >= np.float32(2.0 ** -126):
            scale[i] = s
            codes[i] = np.rint(x[i] / s).astype(np.int8)
    return codes, scale


def numbers(codes, scale):
    """Elements of an 8-bit cache, float64; rows whose scale is not finite are NaN."""
    scale = np.asarray(scale, dtype=np.float64)
    return np.asarray(codes, np.float64) * np.where(np.isfinite(scale), scale, np.nan)[..., None]


def rows(table, tokens, scale):
    """scale * table[token], zeros for a token outside the table."""
    table = np.asarray(table, dtype=np.float64)
    out = np.zeros((len(tokens), table.shape[1]))
    for t, token in enumerate(tokens):
        if 0 <= token < len(table):
            out[t] = float(np.float32(scale)) * table[token]
    return out


def _weights(x, heat):
    """exp(x / heat) of a row, scaled; None if it is no distribution."""
    x = np.asarray(x, dtype=np.float64)
    if np.isnan(x).any() or (x == np.inf).any() or (x == -np.inf).all():
        return None
    if not heat > 0:
        w = np.zeros(len(x))
        w[int(np.argmax(x))] = 1.0
        return w
    return np.exp((x - x.max()) / float(heat))


def verify(logits, tokens, q_start, uniform, drafted=None, temperature=None):
    """(accepted, following) of every conversation."""
    vocab = len(logits[0])
    accepted, following = [], []
    for s in range(len(q_start) - 1):
        first, end = int(q_start[s]), int(q_start[s + 1])
        heat = 1.0 if temperature is None else temperature[s]
        count, token = 0, -1
        for t in range(first, end):
            w = _weights(logits[t], heat)
            if w is None:
                break
            p = w / w.sum()
            rest = p
            if t < end - 1:
                d = int(tokens[t + 1])
                real = 0 <= d < vocab
                q = np.zeros(vocab)
                if drafted is not None and heat > 0:
                    g = _weights(drafted[t], heat)
                    if g is None:
                        break
                    q = g / g.sum()
                    qd = q[d] if real else 0.0
                else:
                    if real:
                        q[d] = 1.0
                    qd = 1.0
                u = 0.5 if not heat > 0 else float(uniform[t][0])
                if real and u * qd < p[d]:
                    count += 1
                    continue
                rest = np.maximum(p - q, 0.0)
                if not rest.sum() > 0:
                    rest = p
            total = np.cumsum(rest)
            above = np.nonzero((total > float(uniform[t][1]) * total[-1]) & (rest > 0))[0]
            token = int(above[0]) if len(above) else int(np.nonzero(rest > 0)[0][-1])
            break
        accepted.append(count)
        following.append(token)
    return np.array(accepted), np.array(following)
