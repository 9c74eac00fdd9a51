"""Cases, inputs and the error bound shared by the grouped-attention GPU tests.

Bound per output element.  Scores: a dot product of D exact 16-bit products
accumulated in fp32 is off by at most 2^-20 of sum |q_i k_i| (the tensor cores'
sums keep at least 23 bits, D <= 128 terms), and the scaling, the cap, the bias
and the subtraction of the running max by a few units of 2^-24 of numbers no
larger than the score or, for a token whose weight matters at all, 48 in log2
units; together dz = 2^-20 (48 + scale max_t sum |q_i k_i|).  Weights: e^dz and
the 16 bits they keep in the product with V, so
  |out - ref| <= (2 dz + 2^-16) sum p |v| / sum p     (call it c),
then one rounding: half a step of the type, eps / 2, of |ref| + c.
"""
import numpy as np

from helpers import to_dev, words
from oracle.grouped import attend
from paged_kv_cache_05_gb300 import workloads as W


def f64(w, dtype):
    return W.words_to_torch(w, dtype).double().numpy()


def make_case(rs, H, HK, D, B, new, ctx, dtype, window=0, qtimes=1.0, wild=True):
    """Host words of a random placement.  Hidden tokens of the used blocks and
    every unused block hold NaN; table entries of blocks that no query of the
    sequence sees are out of the pool (they must not be used)."""
    S = len(ctx)
    need = [-(-c // B) for c in ctx]
    nb, mb = sum(need) + 3, max(max(need), 1) + 1
    perm = rs.permutation(nb)
    nan = np.uint16(0x7E00 if dtype == "f16" else 0x7FC0)
    kc = np.full((nb, HK, B, D), nan, np.uint16)
    vc = np.full((nb, HK, B, D), nan, np.uint16)
    tables = np.full((S, mb), nb + 1000 if wild else -1, np.int32)
    at = 0
    for s in range(S):
        n, m = ctx[s], new[s]
        lo = max(0, n - m - window + 1) if window else 0      # first token any query sees
        for b in range(need[s]):
            phys = perm[at]
            at += 1
            t0 = b * B
            if t0 + B <= lo and m:
                continue
            tables[s, b] = phys
            a, z = max(lo - t0, 0), min(n - t0, B)
            kc[phys, :, a:z] = words((HK, z - a, D), dtype, rs)
            vc[phys, :, a:z] = words((HK, z - a, D), dtype, rs)
    rows = sum(new)
    q = W.torch_to_words((W.words_to_torch(words((max(rows, 1), H, D), dtype, rs), dtype).float()
                          * qtimes).to(W.torch_dtype(dtype)))[:rows]
    qs = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    return dict(q=q, kc=kc, vc=vc, bt=tables, ctx=np.array(ctx, np.int32), qs=qs, H=H, HK=HK, D=D,
                B=B, dtype=dtype, window=window, nb=nb, new=list(new))


def on_device(c):
    import torch
    d = {n: to_dev(c[n], c["dtype"]) for n in ("q", "kc", "vc")}
    d.update(bt=torch.from_numpy(c["bt"]).cuda(), cl=torch.from_numpy(c["ctx"]).cuda(),
             qs=torch.from_numpy(c["qs"]).cuda())
    return d


def reference(c, scale, softcap, slopes):
    """(ref, c of the module's bound)."""
    q, kc, vc = (f64(c[n], c["dtype"]) for n in ("q", "kc", "vc"))
    args = (c["bt"], c["ctx"], c["qs"], scale, softcap, c["window"], slopes)
    ref = attend(q, kc, vc, *args)
    size = attend(q, kc, np.abs(vc), *args)
    live = np.abs(kc[np.isfinite(kc)])
    big = np.abs(q).sum(-1).max() * live.max() if q.size and live.size else 0.0
    # sum |q_i k_i| per pair is far below the product of the sums: take the
    # largest over pairs of a sequence instead where that is affordable
    if q.size and kc.size < 4e6:
        big = 0.0
        for s in range(len(c["ctx"])):
            r = np.abs(q[c["qs"][s]:c["qs"][s + 1]])
            blocks = [b for b in c["bt"][s] if 0 <= b < c["nb"]]
            if r.size and blocks:
                k = np.nan_to_num(np.abs(kc[blocks])).max((0, 2))          # [HK, D]
                G = c["H"] // c["HK"]
                big = max(big, float(np.einsum("rhd,hd->rh", r, np.repeat(k, G, 0)).max()))
    dz = 2.0 ** -20 * (48 + abs(scale) * big)
    return ref, (2 * dz + 2.0 ** -16) * np.abs(size)


def check(got, c, ref, slack, what=""):
    import torch
    g = got.double().cpu().numpy()
    half = torch.finfo(W.torch_dtype(c["dtype"])).eps / 2
    lim = slack + half * (np.abs(ref) + slack) + (2.0 ** -25 if c["dtype"] == "f16" else 0.0)
    assert np.isfinite(g).all(), what
    err = np.abs(g - ref)
    assert (err <= lim).all(), "%s: %d of %d off, worst %g times the bound" % (
        what, (err > lim).sum(), err.size, (err / np.maximum(lim, 1e-30)).max())
