"""Score caps far above the scores, up to caps that change no score, against the
fp64 definition.

Bound: grouped_helpers'.  It holds at every cap when the capped score is as exact,
relative to itself, as the score: cap tanh(z / cap) with a few roundings of 2^-24
and a tanh of 2^-22, all relative, is inside its 2^-20 of scale sum |q_i k_i|.
(An error of 2^-24 of the cap is not: at a cap of 1e8 that is 6 in the score.)  Up
to a cap of 64 the kernels take a form that is off by 2^-20 of the cap: at 64, 2^-14
in the score and 2^-13 of sum p |v| / sum p, which is 2^3 of the bound's 2^-16.
"""
import math

import numpy as np
import pytest

from grouped_helpers import check, make_case, on_device, reference

pytestmark = pytest.mark.gpu

CAPS = [64.0, 65.0, 1e3, 1e5, 1e8, 2e38]


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_05_gb300 import build
    build.build()
    import paged_kv_cache_05_gb300 as m
    return m


def slopes_of(H, biased):
    return (2.0 ** (-8.0 * np.arange(1, H + 1) / H)).astype(np.float32) if biased else None


def direct(cap):
    return 1 + 2.0 ** 3 if cap <= 64 else 1.0


def tensor(a):
    import torch
    return None if a is None else torch.from_numpy(a).cuda()


@pytest.mark.parametrize("cap", CAPS)
@pytest.mark.parametrize("H,HK,D,dtype,biased,window,scale", [
    (6, 2, 64, "f16", False, 0, 0.125), (16, 1, 128, "bf16", True, 700, 0.09),
    (8, 1, 128, "f16", True, 0, -0.3), (12, 1, 64, "bf16", False, 90, 0.125)])
def test_decode(pkv, cap, H, HK, D, dtype, biased, window, scale):
    import torch
    c = make_case(np.random.default_rng(H + D), H, HK, D, 16, [1, 1, 1], [2000, 37, 400], dtype,
                  window, 4.0)
    slopes = slopes_of(H, biased)
    ref, slack = reference(c, scale, cap, slopes)
    slack = slack * direct(cap)
    d = on_device(c)
    out = torch.empty_like(d["q"])
    pkv.paged_attention_decode_grouped(out, d["q"], d["kc"], d["vc"], d["bt"], d["cl"], scale,
                                       softcap=cap, window=window, slopes=tensor(slopes))
    assert pkv.get_device_error() == 0
    check(out, c, ref, slack, "cap %g" % cap)


def test_decode_scores_past_the_cap(pkv):
    """Scores of several times a large cap: the flat ends of the tanh too."""
    import torch
    c = make_case(np.random.default_rng(5), 4, 1, 64, 16, [1, 1], [300, 77], "f16", 0, 30.0)
    for cap, scale in ((100.0, 4.0), (300.0, -2.0)):
        ref, slack = reference(c, scale, cap, None)
        d = on_device(c)
        out = torch.empty_like(d["q"])
        pkv.paged_attention_decode_grouped(out, d["q"], d["kc"], d["vc"], d["bt"], d["cl"], scale,
                                           softcap=cap)
        check(out, c, ref, slack)


def test_decode_cap_of_the_score_range_is_no_cap(pkv):
    """A cap of 1e30 leaves the uncapped call's answer (here within a step)."""
    import torch
    c = make_case(np.random.default_rng(6), 8, 2, 128, 32, [1] * 3, [600, 1, 90], "f16")
    d = on_device(c)
    outs = []
    for cap in (0.0, 1e30):
        out = torch.empty_like(d["q"])
        pkv.paged_attention_decode_grouped(out, d["q"], d["kc"], d["vc"], d["bt"], d["cl"],
                                           1 / math.sqrt(128), softcap=cap)
        outs.append(out.float())
    assert torch.allclose(*outs, rtol=2.0 ** -10, atol=2.0 ** -16)


@pytest.mark.parametrize("cap", CAPS)
@pytest.mark.parametrize("H,HK,D,dtype,new,past,biased,window,scale", [
    (4, 2, 64, "f16", [300, 1, 64], 333, False, 0, 0.125),
    (3, 1, 128, "bf16", [200, 131], 90, True, 150, 0.09),
    (8, 1, 128, "f16", [140], 500, True, 0, -0.3),
    (5, 5, 64, "bf16", [260, 40], 0, False, 100, 0.125)])
def test_prompts(pkv, cap, H, HK, D, dtype, new, past, biased, window, scale):
    prompts(pkv, H, HK, D, dtype, new, past, biased, window, scale, cap)


@pytest.mark.parametrize("cap", CAPS)
@pytest.mark.parametrize("dtype,D,biased", [("f16", 128, False), ("bf16", 64, True)])
def test_prompts_cut_along_the_keys(pkv, cap, dtype, D, biased):
    assert pkv.prefill_grouped_workspace_size(1, 8, 2, D, 16, 300, 6) > 0
    prompts(pkv, 8, 2, D, dtype, [6], 4700, biased, 0, 0.09, cap)


def prompts(pkv, H, HK, D, dtype, new, past, biased, window, scale, cap):
    """fp16 weights keep 11 bits here: 2^-11 of sum p |v| / sum p more (slack is at
    least 2^-16 of that sum), and 2^-25 of the largest |v| a token at most."""
    import torch
    c = make_case(np.random.default_rng(H + D), H, HK, D, 16, new, [n + past for n in new], dtype,
                  window, 4.0)
    slopes = slopes_of(H, biased)
    ref, slack = reference(c, scale, cap, slopes)
    slack = slack * direct(cap)
    if dtype == "f16":
        slack = slack * (1 + 2.0 ** 5) + max(c["ctx"]) * 2.0 ** -25 * 6
    d = on_device(c)
    out = torch.empty_like(d["q"])
    pkv.paged_attention_prefill_grouped(out, d["q"], d["kc"], d["vc"], d["bt"], d["cl"], d["qs"],
                                        scale, max(new), softcap=cap, window=window,
                                        slopes=tensor(slopes))
    assert pkv.get_device_error() == 0
    check(out, c, ref, slack, "cap %g" % cap)
