"""Cases, inputs and the error bound shared by the latent-attention GPU tests.

Bound per output element.  Scores: products of 16-bit values are exact in fp32 and a
sum of D of them is taken 16 at a time, each step off by at most 2^-23 of the partial
sums, so by (D / 16) 2^-23 of sum |q_i k_i| in all; the scaling, the running max and
the exponential by a few units of 2^-24 of numbers no larger than the score or, for a
token whose weight matters at all, 48 in log2 units: dz = (D / 16) 2^-23 scale max_t
sum |q_i k_i| + 2^-20 48.  Weights: e^dz, one rounding to the storage type, at most
half a step, eps / 2, in the products with the values and in their sum alike, and
fp16 weights below 2^-33 of the row's largest lost; so
  |out - ref| <= (2 dz + 2 eps / 2 + n 2^-33) sum p |v| / sum p     (call it c),
then one rounding: half a step of the type, eps / 2, of |ref| + c.
"""
import numpy as np

import oracle.latent as L
from helpers import to_dev, words
from paged_kv_cache_05_gb300 import workloads as W

P = 64


def f64(w, dtype):
    return W.words_to_torch(w, dtype).double().numpy()


def half_step(dtype):
    import torch
    return torch.finfo(W.torch_dtype(dtype)).eps / 2


def nan_word(dtype):
    return np.uint16(0x7E00 if dtype == "f16" else 0x7FC0)


def times(w, dtype, by):
    return W.torch_to_words((W.words_to_torch(w, dtype).float() * by).to(W.torch_dtype(dtype)))


def random_tree(rs, new):
    """Each new token hangs under an earlier one of its sequence or under the cache."""
    bits = []
    for n in new:
        mine = []
        for j in range(n):
            parent = int(rs.randint(-1, j)) if j else -1
            mine.append((mine[parent] if parent >= 0 else 0) | 1 << j)
        bits += mine
    return bits


def to_i64(bits):
    return np.array([b - (1 << 64) if b >= 1 << 63 else b for b in bits], np.int64)


def decode_case(rs, H, R, B, new, ctx, dtype, tree=False, qtimes=1.0):
    """Host words of a random placement.  Slots past a sequence's end and unused blocks
    hold NaN; table entries past a sequence's blocks are out of the pool (they must not
    be used)."""
    S = len(ctx)
    need = [-(-c // B) for c in ctx]
    nb, mb = sum(need) + 3, max(max(need), 1) + 1
    perm = rs.permutation(nb)
    cache = np.full((nb, B, R + P), nan_word(dtype), np.uint16)
    tables = np.full((S, mb), nb + 1000, np.int32)
    at = 0
    for s in range(S):
        for b in range(need[s]):
            phys = perm[at]
            at += 1
            tables[s, b] = phys
            n = min(B, ctx[s] - b * B)
            cache[phys, :n] = words((n, R + P), dtype, rs)
    rows = sum(new)
    q = times(words((max(rows, 1), H, R + P), dtype, rs), dtype, qtimes)[:rows]
    qs = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    return dict(q=q, cache=cache, bt=tables, ctx=np.array(ctx, np.int32), qs=qs, H=H, R=R, B=B,
                dtype=dtype, nb=nb, new=list(new), tree=random_tree(rs, new) if tree else None)


def on_device(c):
    import torch
    d = {n: to_dev(c[n], c["dtype"]) for n in ("q", "cache")}
    d.update(bt=torch.from_numpy(c["bt"]).cuda(), cl=torch.from_numpy(c["ctx"]).cuda(),
             qs=torch.from_numpy(c["qs"]).cuda(),
             tree=None if c["tree"] is None else torch.from_numpy(to_i64(c["tree"])).cuda())
    return d


def run_decode(pkv, c, scale, d=None, **kw):
    import torch
    d = d or on_device(c)
    out = torch.full((c["q"].shape[0], c["H"], c["R"]), 7.0, dtype=W.torch_dtype(c["dtype"]),
                     device="cuda")
    return pkv.latent_attention_decode(out, d["q"], d["cache"], d["bt"], d["cl"], scale,
                                       query_start=d["qs"],
                                       max_query_len=max(c["new"], default=0) or 1,
                                       ancestors=d["tree"], **kw)


def decode_reference(c, scale):
    """(ref, dz of the module's bound)."""
    q, cache = f64(c["q"], c["dtype"]), f64(c["cache"], c["dtype"])
    R = c["R"]
    ref = L.decode(q, cache, c["bt"], c["ctx"], c["qs"], scale, R, c["tree"])
    big = 0.0
    for s, n in enumerate(c["ctx"]):
        blocks = c["bt"][s, :-(-int(n) // c["B"])]
        rows = np.abs(cache[blocks].reshape(-1, R + P)[:n])
        mine = np.abs(q[c["qs"][s]:c["qs"][s + 1]])
        if rows.size and mine.size:
            big = max(big, float((mine @ rows.max(0)).max()))
    dz = (R + P) / 16 * 2.0 ** -23 * abs(scale) * big + 48 * 2.0 ** -20
    return ref, dz


def weighted_size(c, scale):
    """sum p |v| / sum p for every element: the softmax of the scores over |values|."""
    q, cache = f64(c["q"], c["dtype"]), f64(c["cache"], c["dtype"])
    R = c["R"]
    # values beside the keys: rows of R + P keys and R absolute values
    both = np.concatenate([cache, np.abs(cache[..., :R])], -1)
    out = np.zeros(c["q"].shape[:2] + (R,))
    for s, n in enumerate(c["ctx"]):
        n, first, last = int(n), int(c["qs"][s]), int(c["qs"][s + 1])
        if not n or last == first:
            continue
        blocks = c["bt"][s, :-(-n // c["B"])]
        rows = both[blocks].reshape(-1, 2 * R + P)[:n]
        m = last - first
        t = np.arange(n)
        for i in range(m):
            see = t <= n - m + i
            if c["tree"] is not None:
                bits = c["tree"][first + i]
                see = np.array([x < n - m or bool(bits >> int(x - n + m) & 1) for x in t])
            if see.any():
                z = scale * q[first + i] @ rows[see][:, :R + P].T
                out[first + i] = L._softmax(z) @ rows[see][:, R + P:]
    return out


def check(got, ref, dtype, dz, size, n, what=""):
    g = got.double().cpu().numpy()
    half = half_step(dtype)
    slack = (2 * dz + 2 * half + (n * 2.0 ** -33 if dtype == "f16" else 0.0)) * size
    lim = slack + half * (np.abs(ref) + slack) + (2.0 ** -25 if dtype == "f16" else 0.0)
    assert np.isfinite(g).all(), what
    err = np.abs(g - ref)
    assert (err <= lim).all(), "%s: %d of %d off, worst %g times the bound" % (
        what, (err > lim).sum(), err.size, (err / np.maximum(lim, 1e-30)).max())


def check_decode(pkv, c, scale, what="", **kw):
    got = run_decode(pkv, c, scale, **kw)
    assert pkv.get_device_error() == 0, what
    ref, dz = decode_reference(c, scale)
    check(got, ref, c["dtype"], dz, weighted_size(c, scale), max(map(int, c["ctx"]), default=0), what)
    return got


def prefill_case(rs, H, N, new, keys, dtype, qtimes=1.0, pad=8):
    """Host words: keys and values as halves of one tensor, the shared key part as the ends
    of wider rows; rows of no sequence hold NaN."""
    Tq, Tk = sum(new), sum(keys)
    nan = nan_word(dtype)
    up = np.concatenate([words((Tk, H, 2 * N), dtype, rs), np.full((5, H, 2 * N), nan)])
    rows = np.concatenate([words((Tk, pad + P), dtype, rs), np.full((5, pad + P), nan)])
    q = np.concatenate([times(words((Tq, H, N + P), dtype, rs), dtype, qtimes),
                        np.full((3, H, N + P), nan)])
    starts = lambda x: np.concatenate([[0], np.cumsum(x)]).astype(np.int32)  # noqa: E731
    return dict(q=q.astype(np.uint16), up=up.astype(np.uint16), rows=rows.astype(np.uint16),
                qs=starts(new), ks=starts(keys), H=H, N=N, dtype=dtype, new=list(new),
                keys=list(keys), Tq=Tq, pad=pad)


def run_prefill(pkv, c, scale, **kw):
    import torch
    d = {n: to_dev(c[n], c["dtype"]) for n in ("q", "up", "rows")}
    out = torch.full((c["q"].shape[0], c["H"], c["N"]), 7.0, dtype=W.torch_dtype(c["dtype"]),
                     device="cuda")
    pkv.latent_attention_prefill(out, d["q"], d["up"][..., :c["N"]], d["rows"][:, c["pad"]:],
                                 d["up"][..., c["N"]:], torch.from_numpy(c["qs"]).cuda(),
                                 torch.from_numpy(c["ks"]).cuda(), scale,
                                 max(c["new"], default=0), max(c["keys"], default=0), **kw)
    assert (out[c["Tq"]:] == 7.0).all()            # rows of no sequence are left as they were
    return out[:c["Tq"]]


def check_prefill(pkv, c, scale, what="", **kw):
    got = run_prefill(pkv, c, scale, **kw)
    assert pkv.get_device_error() == 0, what
    N, Tk = c["N"], int(c["ks"][-1])
    q, up, rows = (f64(c[n], c["dtype"]) for n in ("q", "up", "rows"))
    q, k, v, r = q[:c["Tq"]], up[:Tk, :, :N], up[:Tk, :, N:], rows[:Tk, c["pad"]:]
    ref = L.prefill(q, k, r, v, c["qs"], c["ks"], scale)
    size = L.prefill(q, k, r, np.abs(v), c["qs"], c["ks"], scale)
    big = 0.0
    for s in range(len(c["new"])):
        a, b = slice(c["qs"][s], c["qs"][s + 1]), slice(c["ks"][s], c["ks"][s + 1])
        if q[a].size and k[b].size:
            most = np.concatenate([np.abs(k[b]).max(0), np.broadcast_to(np.abs(r[b]).max(0), (c["H"], P))], -1)
            big = max(big, float((np.abs(q[a]) * most).sum(-1).max()))
    dz = (N + P) / 16 * 2.0 ** -23 * abs(scale) * big + 48 * 2.0 ** -20
    check(got, ref, c["dtype"], dz, size, max(c["keys"], default=0), what)
    return got
