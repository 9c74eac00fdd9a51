"""The grouped operators' fp64 definitions, pinned: rotation properties and
special cases of the attention that other definitions give."""
import numpy as np
import pytest

import oracle
from helpers import words
from oracle.grouped import attend, norm_rope


def test_rotation_keeps_lengths_and_depends_on_distance_only():
    rs = np.random.default_rng(1)
    f = 10000.0 ** (-np.arange(0, 32, 2) / 32)
    q, k = rs.standard_normal((2, 1, 1, 48))
    dots = []
    for inter in (False, True):
        for p, t in ((7, 3), (1007, 1003)):
            a = norm_rope(q, [p], f, interleaved=inter)
            b = norm_rope(k, [t], f, interleaved=inter)
            assert np.allclose(np.linalg.norm(a), np.linalg.norm(q))
            assert np.array_equal(a[..., 32:], q[..., 32:])
            dots.append(float((a * b).sum()))
        assert abs(dots[-1] - dots[-2]) < 1e-9
    assert np.array_equal(norm_rope(q, [0], f), q)
    # pair i as a complex number times the unit number of its angle
    z = (q[..., 0:32:2] + 1j * q[..., 1:32:2]) * np.exp(1j * 9 * f) * 1.5
    got = norm_rope(q, [9], f, rope_scale=1.5, interleaved=True)
    assert np.allclose(got[..., 0:32:2], z.real) and np.allclose(got[..., 1:32:2], z.imag)


def test_norm_is_the_root_mean_square():
    x = np.array([[[3.0, 4.0]]])
    assert np.allclose(norm_rope(x, [0], [], weight=[1.0, 2.0]), x / np.sqrt(12.5) * [1.0, 2.0])


@pytest.mark.parametrize("H,HK", [(3, 3), (6, 2), (4, 1)])
def test_attention_special_cases(H, HK):
    rs = np.random.default_rng(H * 10 + HK)
    D, B, ctx, new = 64, 8, [19, 1, 0, 8], [5, 1, 0, 8]
    nb = 9
    qs = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    bt = np.array([[4, 0, 7], [2, -1, -1], [-1, -1, -1], [5, -1, -1]], np.int32)
    q, kc, vc = (words(s, "f16", rs) for s in ((14, H, D), (nb, HK, B, D), (nb, HK, B, D)))
    f64 = [w.view(np.float16).astype(np.float64) for w in (q, kc, vc)]
    ref = attend(*f64, bt, ctx, qs, 0.125)
    # every query head with a K/V head of its own: the ungrouped definition
    rep = [np.repeat(w, H // HK, axis=1) for w in (kc, vc)]
    plain = oracle.paged_attention_prefill(q, *rep, bt, np.array(ctx, np.int32), qs, 0.125,
                                           oracle.F16)
    assert np.allclose(ref, plain, rtol=1e-12, atol=1e-12)
    # a window that reaches every token, a cap far above the scores, no slope
    assert np.allclose(attend(*f64, bt, ctx, qs, 0.125, 1e6, 19, np.zeros(H)), ref, atol=1e-9)
    # a window of one token: its own value row
    one = attend(*f64, bt, ctx, qs, 0.125, 5.0, 1, np.ones(H))
    t = 18
    assert np.allclose(one[4], np.repeat(f64[2][bt[0][t // B], :, t % B], H // HK, axis=0))
    # a steep slope leaves the newest token alone
    steep = attend(*f64, bt, ctx, qs, 0.125, 0.0, 0, np.full(H, 1e4))
    assert np.allclose(steep, one)
    # a small cap levels the scores: the mean of the values
    level = attend(*f64, bt, ctx, qs, 0.125, 1e-9)
    assert np.allclose(level[13, 0], f64[2][5, 0].mean(0), atol=1e-8)
