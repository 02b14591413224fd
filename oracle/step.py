"""Embedding rows, low-rank adapters and log probabilities around a step's projections, restated in float64.

TEST INFRASTRUCTURE ONLY (see the package docstring). Plain loops over tokens, adapters and rows, each
formula from its definition.
"""
from __future__ import annotations

import math

import numpy as np


def embed(w_hat, tokens, scale):
    """scale * w_hat[token] per token; zeros for a token outside the matrix."""
    out = np.zeros((len(tokens), w_hat.shape[1]))
    for t, n in enumerate(tokens):
        if 0 <= n < len(w_hat):
            out[t] = scale * w_hat[n]
    return out


def plan(ids, n_adapters, tile, max_tiles):
    """(order, tiles): the tokens of each adapter in turn, and their tiles."""
    order, tiles = [], []
    for a in range(n_adapters):
        mine = [t for t, i in enumerate(ids) if i == a]
        for at in range(0, len(mine), tile):
            tiles.append((a, len(order) + at, min(tile, len(mine) - at), 0))
        order += mine
    order += [-1] * (len(ids) - len(order))
    tiles += [(0, 0, 0, 0)] * (max_tiles - len(tiles))
    return np.array(order, dtype=np.int64), np.array(tiles, dtype=np.int64).reshape(max_tiles, 4)


def lora(y, x, ids, table, scale, a, b):
    """(y + the adapters' parts, S1, S2): per output element the sums of magnitudes that its rounding errors go by,
    S1 = s sum_j |b_jn| sum_k |a_jk x_k| and S2 = s sum_j |h_j b_jn|."""
    out, s1, s2 = y.copy(), np.zeros_like(y), np.zeros_like(y)
    for t, i in enumerate(ids):
        if i < 0:
            continue
        first, r = table[i]
        A, B = a[first:first + r], b[first:first + r]
        h = A @ x[t]
        out[t] += scale[i] * (h @ B)
        s1[t] = abs(scale[i]) * ((np.abs(A) @ np.abs(x[t])) @ np.abs(B))
        s2[t] = abs(scale[i]) * (np.abs(h) @ np.abs(B))
    return out, s1, s2


def order(x):
    """Indices of a row from first to last: larger first, equal ones by index, a NaN as -inf, -0 as 0."""
    v = [(-math.inf if math.isnan(e) else float(e)) for e in x]
    return sorted(range(len(v)), key=lambda i: (-v[i] if v[i] != 0 else 0.0, i))


def logprob(x, scale, token, top):
    """(logprob, rank, lse, entropy, indices, log probabilities) of one row of logits."""
    x = [float(v) for v in x]
    seq = order(x)
    if any(math.isnan(v) or v == math.inf for v in x):
        lp = [math.nan] * len(x)
        lse = entropy = math.nan
    elif all(v == -math.inf for v in x):
        lp, lse, entropy = [-math.inf] * len(x), -math.inf, 0.0
    else:
        z = np.array(x) * scale
        m = z.max()
        e = np.exp(z - m)
        ln_s = math.log(math.fsum(e))
        lp = (z - m) - ln_s
        lse = m + ln_s
        entropy = math.fsum(-math.exp(v) * v for v in lp if v > -math.inf)
    bad = token < 0 or token >= len(x)
    return (0.0 if bad else float(lp[token]), -1 if bad else seq.index(token), lse, entropy,
            seq[:top], [float(lp[i]) for i in seq[:top]])
