"""fp64 definitions of the latent-attention operators, in plain numpy.

TEST INFRASTRUCTURE ONLY, like the rest of this package: values in, values out,
one query row at a time, nothing shared with the CUDA path.
"""
from __future__ import annotations

import numpy as np


def cache_rows(latent, k_rope, positions, inv_freq, weight=None, eps=0.0, rope_scale=1.0,
               interleaved=False):
    """Rows [T, R + P] of latent [T, R] (normed when a weight is given) and k_rope [T, P],
    turned."""
    from .grouped import norm_rope
    x = np.array(latent, np.float64)
    if weight is not None:
        x = x / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    r = norm_rope(np.asarray(k_rope)[:, None], positions, inv_freq, rope_scale=rope_scale,
                  interleaved=interleaved)[:, 0]
    return np.concatenate([x, r], -1)


def _softmax(z):
    e = np.exp(z - z.max(-1, keepdims=True))
    return e / e.sum(-1, keepdims=True)


def decode(q, cache, tables, ctx, query_start, scale, R, ancestors=None):
    """q [rows, H, R + P] over cache [blocks, B, R + P], float64: the rows of a sequence
    are its last tokens; a row attends the tokens up to its own or, with ancestors, those
    before the rows and row j when its bit j is set.  A row that attends nothing is
    zero; rows of no sequence are NaN (not defined)."""
    B = cache.shape[1]
    out = np.full(q.shape[:2] + (R,), np.nan)
    for s, n in enumerate(ctx):
        n, first, last = int(n), int(query_start[s]), int(query_start[s + 1])
        rows = np.concatenate([cache[int(tables[s][t // B])] for t in range(0, n, B)] or
                              [np.zeros((0, q.shape[2]))])[:n]
        m = last - first
        for i in range(m):
            if n == 0:
                out[first + i] = 0.0
                continue
            if ancestors is None:
                see = np.arange(n) <= n - m + i
            else:
                bits = int(ancestors[first + i])
                see = np.array([t < n - m or bits >> (t - n + m) & 1 for t in range(n)], bool)
            if not see.any():
                out[first + i] = 0.0
                continue
            k = rows[see]
            out[first + i] = _softmax(scale * q[first + i] @ k.T) @ k[:, :R]
    return out


def prefill(q, k, k_rope, v, query_start, key_start, scale):
    """The expanded form: q [Tq, H, N + P], k and v [Tk, H, N], k_rope [Tk, P], float64."""
    H, N = k.shape[1:]
    out = np.full((q.shape[0], H, N), np.nan)
    for s in range(len(query_start) - 1):
        q0, q1, k0, k1 = (int(x) for x in (query_start[s], query_start[s + 1], key_start[s],
                                           key_start[s + 1]))
        for i in range(q1 - q0):
            end = k1 - (q1 - q0) + i + 1
            for h in range(H):
                z = k[k0:end, h] @ q[q0 + i, h, :N] + k_rope[k0:end] @ q[q0 + i, h, N:]
                out[q0 + i, h] = _softmax(scale * z) @ v[k0:end, h]
    return out
