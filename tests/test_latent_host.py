"""Host side of the latent entry points (no GPU): argument checks of the C ABI, workspace
sizes, and pins of the fp64 definitions."""
import ctypes

import numpy as np
import pytest

import oracle.latent as L
import paged_kv_cache_05_gb300 as pkv
from oracle.grouped import norm_rope


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_cache_05_gb300 import build
    build.build()


def refused(fn, names, good, **kw):
    lib = pkv.lib()
    a = dict(zip(names, good))
    assert set(kw) <= set(a), kw
    a.update(kw)
    return getattr(lib, fn)(*[a[n] for n in names])


PTR = 4096                                         # an aligned address, never dereferenced
WRITE = ("qo qos qoh q qs qh l ls r rs cache slots pos ph inter rscale w eps T H R P B nb dt st".split(),
         [PTR, 256, 64, PTR + 8192, 256, 64, PTR + 16384, 320, PTR + 32768, 320, PTR << 8, PTR, PTR, PTR,
          0, 1.0, None, 1e-6, 2, 4, 256, 64, 16, 4, 0, None])
GATHER = ("rows cache bt ks S R P B mb nb T dt st".split(),
          [PTR, PTR << 8, PTR, PTR, 2, 256, 64, 16, 4, 9, 5, 0, None])
PROMPT = ("out q qs qh k ks kh r rs v vs vh qst kst scale S H N P mq mk Tq Tk dt ws wb st".split(),
          [PTR << 8, PTR, 768, 192, PTR, 512, 128, PTR, 64, PTR, 512, 128, PTR, PTR, 0.1, 1, 4, 128, 64,
           2, 4, 2, 4, 0, None, 0, None])
DECODE = ("out q cache bt cl qs an scale S H R P B mb nb mq T dt ws wb st".split(),
          [PTR << 8, PTR, PTR << 10, PTR, PTR, PTR, None, 0.1, 2, 4, 256, 64, 16, 4, 9, 2, 3, 0, PTR << 12,
           1 << 30, None])


@pytest.mark.parametrize("fn,spec,bad", [
    ("pkv_latent_norm_rope_and_cache", WRITE, [
        dict(R=128), dict(R=576), dict(P=32), dict(B=12), dict(nb=0), dict(nb=1 << 60), dict(dt=7),
        dict(H=0), dict(T=-1), dict(T=1 << 29), dict(eps=-1.0), dict(eps=float("nan")),
        dict(rscale=float("inf")), dict(qs=100), dict(qs=250), dict(qh=60), dict(qoh=65), dict(ls=64),
        dict(rs=60), dict(ls=(1 << 32) + 8), dict(q=None), dict(ph=None), dict(slots=PTR + 4),
        dict(q=PTR + 8200), dict(w=PTR + 4), dict(l=PTR), dict(cache=PTR), dict(cache=PTR + 16384)]),
    ("pkv_gather_latent", GATHER, [
        dict(R=300), dict(P=0), dict(B=1), dict(nb=0), dict(S=-1), dict(S=65536), dict(mb=0), dict(T=-1),
        dict(rows=None), dict(ks=PTR + 2), dict(rows=PTR + 8), dict(rows=PTR << 8), dict(dt=-1)]),
    ("pkv_latent_attention_prefill", PROMPT, [
        dict(N=96), dict(P=32), dict(S=-1), dict(H=0), dict(mq=-1), dict(mk=-1), dict(Tq=-1),
        dict(Tq=(1 << 30) + 1), dict(dt=2), dict(scale=float("nan")), dict(scale=3e38), dict(qs=700),
        dict(qh=128), dict(kh=60), dict(ks=516), dict(vs=1), dict(rs=8), dict(out=None), dict(r=None),
        dict(k=PTR + 2), dict(kst=PTR + 1), dict(out=PTR), dict(mk=513), dict(mk=513, ws=PTR + 8),
        dict(mk=513, ws=PTR << 12, wb=100), dict(mk=513, ws=PTR << 8, wb=1 << 40)]),
    ("pkv_latent_attention_decode", DECODE, [
        dict(R=320), dict(P=128), dict(S=-1), dict(S=16385), dict(H=0), dict(H=70000), dict(B=128),
        dict(mb=0), dict(mb=1 << 28), dict(nb=0), dict(nb=1 << 27), dict(mq=-1), dict(T=-1),
        dict(T=1 << 30), dict(dt=9), dict(scale=float("inf")), dict(qs=None), dict(an=PTR, mq=65),
        dict(an=PTR + 4), dict(cl=PTR + 1), dict(q=None), dict(ws=None), dict(ws=PTR + 16), dict(wb=0),
        dict(out=PTR + 2), dict(out=PTR), dict(out=PTR << 10), dict(out=PTR << 12)]),
])
def test_arguments_are_checked(fn, spec, bad):
    for kw in bad:
        assert refused(fn, *spec, **kw) == 1, (fn, kw)
        assert fn in pkv.pagedkv.last_error()


def test_empty_calls_are_accepted():
    assert refused("pkv_latent_norm_rope_and_cache", *WRITE, T=0) == 0
    assert refused("pkv_gather_latent", *GATHER, T=0) == 0
    assert refused("pkv_latent_attention_prefill", *PROMPT, Tq=0) == 0
    assert refused("pkv_latent_attention_decode", *DECODE, S=0, T=0) == 0


def test_workspace_sizes():
    one = pkv.latent_decode_workspace_size(64, 16, 512)
    assert one < pkv.latent_decode_workspace_size(64, 128, 512)
    # a tile has 128 rows at most
    assert pkv.latent_decode_workspace_size(64, 128, 512) == pkv.latent_decode_workspace_size(9, 200, 512, 7)
    assert pkv.latent_decode_workspace_size(64, 16, 256) < one
    assert pkv.latent_prefill_workspace_size(128, 2000, 512) == 0
    assert pkv.latent_prefill_workspace_size(64, 2000, 513) < pkv.latent_prefill_workspace_size(128, 2000, 513)
    assert pkv.latent_prefill_workspace_size(128, 512, 9000) == pkv.latent_prefill_workspace_size(128, 9000, 9000)
    n = ctypes.c_size_t(0)
    for a in ((1, 0, 512, 1), (1, 1, 100, 1), (-1, 1, 512, 1), (1, 1, 512, -1)):
        assert pkv.lib().pkv_latent_decode_workspace_size(*a, ctypes.byref(n)) == 1
    assert pkv.lib().pkv_latent_prefill_workspace_size(96, 1, 1, ctypes.byref(n)) == 1


def test_definitions():
    """The absorbed form is the expanded one; a chain is a tree of one branch."""
    rs = np.random.RandomState(0)
    R, P, N, H, n, m, B = 12, 4, 6, 3, 11, 4, 4
    rows = rs.standard_normal((n, R + P))
    up_k, up_v = rs.standard_normal((2, H, N, R))
    q = rs.standard_normal((m, H, N + P))
    cache = np.zeros((4, B, R + P))
    tables = np.array([[2, 0, 3, -1]])
    for t in range(n):
        cache[tables[0, t // B], t % B] = rows[t]
    full = np.concatenate([np.einsum("thn,hnr->thr", q[..., :N], up_k), q[..., N:]], -1)
    chain = [(1 << i + 1) - 1 for i in range(m)]
    a = L.decode(full, cache, tables, [n], [0, m], 0.3, R)
    assert np.allclose(a, L.decode(full, cache, tables, [n], [0, m], 0.3, R, chain))
    k = np.einsum("tr,hnr->thn", rows[:, :R], up_k)
    v = np.einsum("tr,hnr->thn", rows[:, :R], up_v)
    b = L.prefill(q, k, rows[:, R:], v, [0, m], [0, n], 0.3)
    assert np.allclose(np.einsum("thr,hnr->thn", a, up_v), b)
    # by hand: the last row over all keys, head 1
    z = 0.3 * np.array([k[t, 1] @ q[-1, 1, :N] + rows[t, R:] @ q[-1, 1, N:] for t in range(n)])
    w = np.exp(z) / np.exp(z).sum()
    assert np.allclose(b[-1, 1], w @ v[:, 1])
    assert (L.decode(full, cache, tables, [m], [0, m], 0.3, R, [0] * m) == 0).all()
    # rows of the cache: norm of the latent, rotation of the shared part alone
    pos, freq = np.arange(5), np.array([0.7, 0.1])
    got = L.cache_rows(rows[:5, :R], rows[:5, R:], pos, freq, np.ones(R), 0.0)
    assert np.allclose((got[:, :R] ** 2).mean(-1), 1)
    assert np.allclose(got[:, R:], norm_rope(rows[:5, None, R:], pos, freq)[:, 0])
