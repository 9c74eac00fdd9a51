"""fp64 definitions of the grouped-head operators, in plain numpy.

TEST INFRASTRUCTURE ONLY, like the rest of this package: values in, values out,
one query row at a time, nothing shared with the CUDA path.
"""
from __future__ import annotations

import numpy as np


def norm_rope(x, positions, inv_freq, weight=None, eps=0.0, rope_scale=1.0, interleaved=False):
    """Rows x [T, H, D] (float64) normed per head (when a weight is given) and
    turned by positions [T] * inv_freq [rot / 2]."""
    x = np.array(x, dtype=np.float64)
    if weight is not None:
        x = x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    out = x.copy()
    n = len(inv_freq)
    for i in range(n):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
        angle = np.asarray(positions, np.float64) * float(inv_freq[i])
        c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
        out[..., a] = rope_scale * (x[..., a] * c - x[..., b] * s)
        out[..., b] = rope_scale * (x[..., b] * c + x[..., a] * s)
    return out


def attend(q, kc, vc, tables, ctx, query_start, scale, softcap=0.0, window=0, slopes=None):
    """Causal attention of each sequence's new rows over its paged K/V, all
    float64: q [rows, H, D], pools [blocks, HK, B, D].  Query row i of a sequence
    with n tokens and m new ones is at position p = n - m + i and attends the
    positions t <= p (t > p - window when window > 0) with the scores
    z = scale q.k;  z = softcap tanh(z / softcap) when softcap > 0;
    z += slopes[h] (t - p) when slopes are given.  Query head h reads K/V head
    h // (H // HK).  A row that attends nothing is zero; rows of no sequence are
    NaN (not defined)."""
    rows, H, D = q.shape
    HK, B = kc.shape[1], kc.shape[2]
    out = np.full((rows, H, D), np.nan)
    for s, n in enumerate(ctx):
        n = int(n)
        first, last = int(query_start[s]), int(query_start[s + 1])
        if last == first:
            continue
        # the blocks that hold a token some row sees
        seen = max(0, n - (last - first) - window + 1) if window > 0 else 0
        base = seen // B * B
        blocks = [int(tables[s][t // B]) for t in range(base, n, B)]
        if n:
            k = np.concatenate([kc[b] for b in blocks], axis=1)
            v = np.concatenate([vc[b] for b in blocks], axis=1)
        for r in range(first, last):
            p = n - (last - first) + (r - first)
            lo = max(0, p - window + 1) if window > 0 else 0
            if p < lo:
                out[r] = 0.0
                continue
            for h in range(H):
                g = h // (H // HK)
                z = k[g, lo - base:p + 1 - base] @ q[r, h] * scale
                if softcap > 0:
                    z = softcap * np.tanh(z / softcap)
                if slopes is not None:
                    z = z + float(slopes[h]) * (np.arange(lo, p + 1) - p)
                e = np.exp(z - z.max())
                out[r, h] = (e @ v[g, lo - base:p + 1 - base]) / e.sum()
    return out
