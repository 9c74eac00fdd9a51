"""Rotation frequencies and the argument checks of the norm-rotate-write call,
without a GPU."""
import math

import numpy as np
import pytest


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_05_gb300 import build
    build.build()
    import paged_kv_cache_05_gb300 as m
    return m


def test_frequencies(pkv):
    i = np.arange(32)
    plain, one = pkv.rope_inv_freq(64, 10000.0)
    assert one == 1.0 and np.allclose(plain, 10000.0 ** (-2 * i / 64), rtol=1e-14)
    lin, one = pkv.rope_inv_freq(64, 10000.0, "linear", 4.0)
    assert one == 1.0 and np.allclose(lin, plain / 4, rtol=1e-14)
    base, one = pkv.rope_inv_freq(64, 10000.0, "base", 4.0)
    assert one == 1.0 and math.isclose(base[0], 1.0)
    assert math.isclose(base[-1], plain[-1] / 4, rel_tol=1e-12)     # the slowest: the whole factor
    assert (np.diff(base / plain) < 0).all()
    parts, scale = pkv.rope_inv_freq(64, 10000.0, "by_parts", 4.0, 4096, 32.0, 1.0)
    assert math.isclose(scale, 0.1 * math.log(4) + 1, rel_tol=1e-6)
    turns = 4096 * plain / (2 * math.pi)
    assert np.allclose(parts[turns > 40], plain[turns > 40])        # fast pairs kept
    assert np.allclose(parts[turns < 0.8], plain[turns < 0.8] / 4)  # slow ones by the factor
    ratio = plain / parts
    assert (np.diff(ratio) >= -1e-12).all() and ratio.min() >= 1 - 1e-12 and ratio.max() <= 4 + 1e-12
    same, one = pkv.rope_inv_freq(64, 10000.0, "by_parts", 1.0, 4096)
    assert one == 1.0 and np.allclose(same, plain, rtol=1e-14)


def test_frequencies_refused(pkv):
    bad = [dict(rot_dim=7), dict(rot_dim=0), dict(base=1.0), dict(base=float("nan")),
           dict(scaling="linear", factor=0.5), dict(scaling="base", factor=float("inf")),
           dict(rot_dim=2, scaling="base", factor=2.0), dict(scaling="by_parts", factor=2.0),
           dict(scaling="by_parts", factor=2.0, original_len=100, beta_fast=1.0, beta_slow=2.0)]
    for kw in bad:
        with pytest.raises(pkv.PagedKVError) as e:
            pkv.rope_inv_freq(**dict(dict(rot_dim=64), **kw))
        assert e.value.status == 1
    with pytest.raises(ValueError):
        pkv.rope_inv_freq(64, scaling="other")


def test_phases(pkv):
    """2^64 turns make no turn: phases are exact binary fractions, negative and
    large frequencies wrap, and no frequency rounds up to a whole turn."""
    two_pi = 6.283185307179586
    f = np.array([0.0, two_pi / 4, two_pi * 1.5, -two_pi / 4, -1e-300, 1.0, 1e9])
    p = pkv.rope_phases(f, "cpu").numpy().view(np.uint64)
    assert p[0] == 0 and p[1] == 1 << 62 and p[2] == 1 << 63 and p[3] == 3 << 62 and p[4] == 0
    assert abs(float(p[5]) / 2.0 ** 64 - 1 / two_pi) < 1e-15
    assert abs(float(p[6]) / 2.0 ** 64 - (1e9 / two_pi) % 1.0) < 1e-7
    with pytest.raises(pkv.PagedKVError):
        pkv.rope_phases([1.0, float("inf")], "cpu")
    assert pkv.rope_phases([], "cpu").numel() == 0


def test_bad_arguments_are_refused_before_any_gpu_call(pkv):
    L = pkv.lib()
    a = 1 << 40                       # never dereferenced
    gap = 1 << 32
    names = ["q_out", "q", "k", "v", "qs", "ks", "vs", "kc", "vc", "slots", "pos", "ph", "rot",
             "inter", "rscale", "qw", "kw", "eps", "T", "H", "HK", "D", "B", "nb", "dtype", "stream"]
    base = [a, a + gap, a + 2 * gap, a + 3 * gap, 512, 128, 128, a + 4 * gap, a + 5 * gap,
            a + 6 * gap, a + 7 * gap, a + 8 * gap, 64, 0, 1.0, None, None, 1e-6, 4, 8, 2, 64, 16,
            64, 0, None]

    def call(**kw):
        args = list(base)
        for k, v in kw.items():
            args[names.index(k)] = v
        return L.pkv_norm_rope_and_cache(*args)

    for kw in [dict(H=0), dict(HK=0), dict(D=96), dict(B=12), dict(nb=0), dict(dtype=2),
               dict(rot=60), dict(rot=72), dict(rot=-8), dict(rscale=float("nan")),
               dict(eps=-1.0), dict(eps=float("inf")), dict(T=-1), dict(T=(1 << 28) + 1),
               dict(qs=504), dict(ks=120), dict(vs=132), dict(q_out=None), dict(v=None),
               dict(slots=None), dict(pos=None), dict(ph=None), dict(q=a + gap + 8),
               dict(kc=a + 4 * gap + 2), dict(qw=a + 4), dict(slots=a + 4), dict(pos=a + 2),
               dict(q_out=a + gap, qs=520),                       # in place, rows apart
               dict(q_out=a + gap + 16), dict(k=a), dict(v=a + 1024),
               dict(kc=a), dict(vc=a + gap), dict(vc=a + 4 * gap + 1024)]:
        assert call(**kw) == 1, kw
        assert "pkv_norm_rope_and_cache" in pkv.pagedkv.last_error()
    assert call(T=0) == 0
