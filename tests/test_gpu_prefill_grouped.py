"""The prompt phase with shared K/V heads, capped scores, windows and biases,
against the fp64 definition.

Bound: grouped_helpers', with the weights' own rounding of this kernel: fp16
weights are rounded to 11 bits (relative 2^-11, and 2^-25 below the normal
range, each of at most ctx tokens, against a sum of weights of at least 1);
bf16 weights keep 16 bits as there.
"""
import math

import numpy as np
import pytest

from grouped_helpers import check, f64, make_case, on_device, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_05_gb300 import build
    build.build()
    import paged_kv_cache_05_gb300 as m
    return m


def alibi(H):
    return (2.0 ** (-8.0 * np.arange(1, H + 1) / H)).astype(np.float32)


def bounded(c, scale, cap, slopes):
    ref, slack = reference(c, scale, cap, slopes)
    if c["dtype"] == "f16":
        v = np.abs(f64(c["vc"], "f16"))
        top = v[np.isfinite(v)].max() if np.isfinite(v).any() else 0.0
        # slack is (2 dz + 2^-16) A with A = sum p |v| / sum p: A <= slack 2^16
        size = slack / (2.0 ** -16)
        slack = slack + np.minimum(size, top) * 2.0 ** -11 + int(c["ctx"].max()) * 2.0 ** -25 * top
    return ref, slack


def run(pkv, c, d, scale, cap=0.0, slopes=None, most=None, **kw):
    import torch
    rows = c["q"].shape[0]
    out = torch.full((rows + 3, c["H"], c["D"]), 7.0, dtype=d["q"].dtype, device="cuda")
    sl = None if slopes is None else torch.from_numpy(slopes).cuda()
    pkv.paged_attention_prefill_grouped(out[:rows], d["q"], d["kc"], d["vc"], d["bt"], d["cl"],
                                        d["qs"], scale, most or max(max(c["new"]), 1), softcap=cap,
                                        window=c["window"], slopes=sl, **kw)
    assert (out[rows:] == 7.0).all()
    return out[:rows]


WHOLE = [1, 5, 127, 128, 129, 0, 255, 256, 257, 300]
CASES = [
    # H, HK, D, B, dtype, new, past, window, softcap, biased
    (8, 8, 128, 16, "f16", WHOLE, 0, 0, 0.0, False),
    (8, 2, 128, 16, "bf16", WHOLE, 0, 0, 0.0, False),
    (6, 3, 64, 8, "f16", WHOLE, 0, 0, 0.0, True),
    (5, 1, 64, 32, "bf16", WHOLE, 0, 0, 30.0, False),
    (3, 1, 128, 64, "f16", WHOLE, 0, 0, 20.0, True),
    (4, 1, 128, 16, "bf16", [300, 1, 64], 700, 0, 0.0, False),
    (4, 2, 64, 16, "f16", [300, 1, 64, 513], 700, 100, 0.0, False),
    (4, 2, 128, 8, "bf16", [300, 1, 64, 513], 333, 128, 50.0, False),
    (2, 1, 128, 64, "f16", [260, 700], 900, 129, 0.0, True),
    (7, 7, 64, 64, "bf16", [600], 77, 1, 0.0, False),
    (2, 2, 64, 16, "f16", [1000], 0, 300, 5.0, True),
    (1, 1, 128, 16, "bf16", [513], 1, 256, 0.0, False),
    (16, 2, 64, 8, "bf16", [1] * 9, 40, 0, 0.0, False),
    (2, 1, 64, 32, "f16", [700], 2000, 2000, 0.0, False),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "%dx%d-D%d-B%d-%s-new%d-past%d-w%d-c%g-%d" % (
    c[0], c[1], c[2], c[3], c[4], max(c[5]), c[6], c[7], c[8], c[9]))
def test_against_fp64(pkv, case):
    H, HK, D, B, dtype, new, past, window, cap, biased = case
    rs = np.random.default_rng(H * 100 + D + B + past + window)
    ctx = [n + (past - 13 * i if past > 13 * i else 0) if n else 0 for i, n in enumerate(new)]
    c = make_case(rs, H, HK, D, B, new, ctx, dtype, window, 6.0 if cap else 1.0)
    slopes = alibi(H) if biased else None
    scale = 1 / math.sqrt(D)
    ref, slack = bounded(c, scale, cap, slopes)
    d = on_device(c)
    out = run(pkv, c, d, scale, cap, slopes)
    assert pkv.get_device_error() == 0
    check(out, c, ref, slack)


def test_equals_the_plain_entry_point_without_sharing(pkv):
    """With one K/V head per query head and nothing else asked for, the same
    bits as pkv_paged_attention_prefill."""
    import torch
    for dtype, D in (("f16", 128), ("bf16", 64)):
        c = make_case(np.random.default_rng(2), 4, 4, D, 16, [300, 20], [900, 20], dtype,
                      wild=False)
        d = on_device(c)
        out = run(pkv, c, d, 0.1)
        want = torch.empty_like(d["q"])
        pkv.paged_attention_prefill(want, d["q"], d["kc"], d["vc"], d["bt"], d["cl"], d["qs"], 0.1,
                                    300)
        assert torch.equal(out.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("scale", [0.0, -0.3])
@pytest.mark.parametrize("cap,biased", [(0.0, False), (10.0, False), (0.0, True), (10.0, True)])
def test_scales(pkv, scale, cap, biased):
    c = make_case(np.random.default_rng(3), 4, 2, 64, 16, [200, 150], [200, 450], "bf16", 170)
    slopes = np.array([-0.25, 0.0, 0.5, -1.0], np.float32) if biased else None
    ref, slack = bounded(c, scale, cap, slopes)
    check(run(pkv, c, on_device(c), scale, cap, slopes), c, ref, slack)


def test_bad_inputs_are_flagged(pkv):
    from paged_kv_cache_05_gb300.pagedkv import DEVERR_BAD_BLOCK, DEVERR_BAD_CONTEXT
    import torch
    c = make_case(np.random.default_rng(6), 4, 2, 64, 16, [40, 90, 20], [40, 90, 20], "f16",
                  wild=False)
    ref, slack = bounded(c, 0.125, 0.0, None)
    d = on_device(c)
    d["kc"].nan_to_num_(0.0)
    d["vc"].nan_to_num_(0.0)
    d["bt"][1, 2] = -5
    out = run(pkv, c, d, 0.125)
    assert pkv.get_device_error() == DEVERR_BAD_BLOCK and pkv.get_device_error() == 0
    keep = np.r_[0:40, 130:150]
    check(out[torch.from_numpy(keep).cuda()], c, ref[keep], slack[keep])
    d["bt"][1, 2] = 0
    d["cl"][1] = 1 << 30
    out = run(pkv, c, d, 0.125)
    assert pkv.get_device_error() == DEVERR_BAD_CONTEXT
    check(out[torch.from_numpy(keep).cuda()], c, ref[keep], slack[keep])
    assert (out[40:130] == 7.0).all()                     # that sequence was skipped


def test_captured_and_replayed(pkv):
    import torch
    c = make_case(np.random.default_rng(8), 8, 2, 128, 16, [140, 33], [700, 33], "f16", 200,
                  wild=False)
    d = on_device(c)
    out = torch.empty_like(d["q"])
    call = lambda o, s=None: pkv.paged_attention_prefill_grouped(  # noqa: E731
        o, d["q"], d["kc"], d["vc"], d["bt"], d["cl"], d["qs"], 0.09, 140, softcap=20.0,
        window=200, stream=s)
    call(out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out)
    side = torch.cuda.Stream()
    for k in range(2):
        d["q"].mul_(1.5)
        out.zero_()
        graph.replay()
        want = torch.empty_like(out)
        torch.cuda.synchronize()
        call(want, side)
        side.synchronize()
        assert torch.equal(out, want)


def test_pool_past_32_bit_offsets(pkv):
    import torch
    HK, B, D, H = 8, 16, 128, 16
    nb = (1 << 32) // (HK * B * D) + 50
    kc = torch.zeros((nb, HK, B, D), dtype=torch.float16, device="cuda")
    vc = torch.zeros((nb, HK, B, D), dtype=torch.float16, device="cuda")
    c = make_case(np.random.default_rng(9), H, HK, D, B, [37, 10], [37, 300], "f16", wild=False)
    d = on_device(c)
    far = nb - c["nb"]
    kc[far:], vc[far:] = d["kc"], d["vc"]
    ref, slack = bounded(c, 0.09, 0.0, None)
    out = torch.empty_like(d["q"])
    pkv.paged_attention_prefill_grouped(out, d["q"], kc, vc, d["bt"] + far, d["cl"], d["qs"], 0.09,
                                        37)
    assert pkv.get_device_error() == 0
    check(out, c, ref, slack)


def test_a_serving_run(pkv):
    """The three operators as a server calls them: prompts normed, turned and
    written, attended; then tokens one at a time, in blocks the manager gives;
    each step against the fp64 definitions on the values held in the cache."""
    import torch
    from helpers import to_dev, words
    from oracle.grouped import attend, norm_rope
    from paged_kv_cache_05_gb300 import workloads as W
    rs = np.random.default_rng(77)
    H, HK, D, B, dtype, nb, window, cap = 8, 2, 64, 16, "bf16", 80, 90, 25.0
    prompts = [130, 17, 64]
    bm = pkv.BlockManager(nb, B, 5)
    kc = torch.full((nb, HK, B, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    vc = kc.clone()
    f, rscale = pkv.rope_inv_freq(32, 10000.0, "by_parts", 4.0, 64)
    ph = pkv.rope_phases(f)
    qw, kw = (torch.from_numpy((1 + 0.2 * rs.standard_normal(D)).astype(np.float32)).cuda()
              for _ in range(2))
    scale = 1 / math.sqrt(D)

    def step(slots, positions, new, decode):
        T = len(slots)
        qkv = to_dev(words((T, H + 2 * HK, D), dtype, rs), dtype)
        q, k, v = qkv[:, :H], qkv[:, H:H + HK], qkv[:, H + HK:]
        turned = torch.empty((T, H, D), dtype=torch.bfloat16, device="cuda")
        pkv.norm_rope_and_cache(turned, q, k, v, kc, vc, torch.from_numpy(slots).cuda(),
                                torch.from_numpy(positions).cuda(), ph, qw, kw, 1e-6, rscale)
        ref_q = norm_rope(q.double().cpu().numpy(), positions, f, qw.cpu().numpy(), 1e-6, rscale)
        assert np.allclose(turned.double().cpu().numpy(), ref_q, rtol=2.0 ** -8, atol=1e-5)
        bt, ctx = bm.export([0, 1, 2], 20)
        qs = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        t = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
        out = torch.empty_like(turned)
        if decode:
            pkv.paged_attention_decode_grouped(out, turned, kc, vc, t(bt), t(ctx), scale, cap,
                                               window)
        else:
            pkv.paged_attention_prefill_grouped(out, turned, kc, vc, t(bt), t(ctx), t(qs), scale,
                                                max(new), cap, window)
        assert pkv.get_device_error() == 0
        c = dict(q=W.torch_to_words(turned), kc=W.torch_to_words(kc), vc=W.torch_to_words(vc),
                 bt=bt, ctx=ctx, qs=qs, H=H, HK=HK, D=D, B=B, dtype=dtype, window=window, nb=nb,
                 new=new)
        ref, slack = reference(c, scale, cap, None)
        check(out, c, ref, slack)

    slots = [bm.add_sequence(i, n) for i, n in enumerate(prompts)]
    step(np.concatenate(slots), np.concatenate([np.arange(n) for n in prompts]).astype(np.int32),
         prompts, False)
    for k in range(20):
        s, pairs = bm.append_slots([0, 1, 2])
        assert len(pairs) == 0
        step(s, np.array([n + k for n in prompts], np.int32), [1, 1, 1], True)


@pytest.mark.parametrize("S,H,HK", [(400, 2, 1), (300, 6, 2), (3, 4, 4)])
def test_many_short_prompts_and_many_items(pkv, S, H, HK):
    """More sequences than threads of a block, more items than a dealt batch
    holds, more units than its rounds: the schedule by runs, packed and not."""
    rs = np.random.default_rng(S)
    new = [1 + i % 7 for i in range(S)] if S > 3 else [3000, 2500, 129]
    c = make_case(rs, H, HK, 64, 8, new, [n + i % 3 for i, n in enumerate(new)], "bf16",
                  0 if S > 3 else 40)
    ref, slack = bounded(c, 0.125, 0.0, None)
    check(run(pkv, c, on_device(c), 0.125), c, ref, slack)
    assert pkv.get_device_error() == 0


def test_rows_past_max_query_len_are_flagged(pkv):
    from paged_kv_cache_05_gb300.pagedkv import DEVERR_BAD_CONTEXT
    c = make_case(np.random.default_rng(12), 4, 2, 64, 16, [300, 20], [300, 20], "f16",
                  wild=False)
    ref, slack = bounded(c, 0.125, 0.0, None)
    out = run(pkv, c, on_device(c), 0.125, most=128)
    assert pkv.get_device_error() == DEVERR_BAD_CONTEXT
    check(out[:128], c, ref[:128], slack[:128])
    check(out[300:], c, ref[300:], slack[300:])
    assert (out[256:300] == 7.0).all()
