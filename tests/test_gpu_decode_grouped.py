"""Decode attention with shared K/V heads, capped scores, windows and biases,
against the fp64 definition (bound: grouped_helpers)."""
import math

import numpy as np
import pytest

from grouped_helpers import check, make_case, on_device, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_05_gb300 import build
    build.build()
    import paged_kv_cache_05_gb300 as m
    return m


def alibi(H):
    return (2.0 ** (-8.0 * np.arange(1, H + 1) / H)).astype(np.float32)


def run(pkv, c, d, scale, softcap=0.0, slopes=None, **kw):
    import torch
    out = torch.full((len(c["ctx"]) + 1, c["H"], c["D"]), 7.0, dtype=d["q"].dtype, device="cuda")
    sl = None if slopes is None else torch.from_numpy(slopes).cuda()
    pkv.paged_attention_decode_grouped(out[:-1], d["q"], d["kc"], d["vc"], d["bt"], d["cl"], scale,
                                       softcap=softcap, window=c["window"], slopes=sl, **kw)
    assert (out[-1] == 7.0).all()                        # the row behind the last sequence
    return out[:-1]


CTX = [0, 1, 7, 8, 15, 16, 17, 31, 33, 63, 64, 65, 100, 255, 0, 300]
CASES = [
    # H, HK, D, B, dtype, ctx, window, softcap, biased
    (8, 8, 128, 16, "f16", CTX, 0, 0.0, False),
    (4, 4, 64, 8, "bf16", CTX, 0, 0.0, True),
    (32, 8, 128, 16, "bf16", CTX, 0, 0.0, False),
    (6, 2, 64, 32, "f16", CTX, 0, 30.0, False),
    (40, 8, 128, 8, "f16", CTX, 17, 0.0, False),
    (8, 1, 128, 64, "bf16", CTX, 64, 20.0, True),
    (24, 2, 128, 16, "bf16", CTX, 0, 0.0, True),         # 12 heads a K/V head
    (16, 1, 64, 64, "f16", CTX, 1, 0.0, False),
    (71, 1, 64, 16, "f16", CTX, 100, 50.0, True),        # 5 rows of 16, 16, 16, 16 and 7
    (34, 2, 128, 32, "bf16", CTX, 33, 0.0, False),       # 17 heads: 16 and 1
    (3, 1, 128, 8, "f16", [1], 0, 0.0, False),
    (8, 2, 64, 16, "bf16", [0, 0, 0], 0, 0.0, False),
    (8, 2, 64, 8, "bf16", [4097, 2500, 1], 0, 0.0, True),
    (10, 2, 128, 16, "f16", [5000, 33, 1777], 1500, 0.0, False),
    (2, 1, 128, 16, "bf16", [9000], 0, 5.0, False),      # one row over many ranges
    (4, 2, 64, 64, "f16", [3 + 5 * (i % 41) for i in range(300)], 0, 0.0, False),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "%dx%d-D%d-B%d-%s-S%d-w%d-c%g-%d" % (
    c[0], c[1], c[2], c[3], c[4], len(c[5]), c[6], c[7], c[8]))
def test_against_fp64(pkv, case):
    H, HK, D, B, dtype, ctx, window, cap, biased = case
    rs = np.random.default_rng(H * 1000 + D + B + len(ctx) + window)
    c = make_case(rs, H, HK, D, B, [1 if n else 0 for n in ctx], ctx, dtype, window,
                  6.0 if cap else 1.0)
    # a query row per sequence, the empty ones' too
    from helpers import words
    full = words((len(ctx), H, D), dtype, rs)
    full[np.array(ctx) > 0] = c["q"]
    slopes = alibi(H) if biased else None
    scale = 1 / math.sqrt(D)
    ref_live, slack_live = reference(c, scale, cap, slopes)
    ref, slack = np.zeros((len(ctx), H, D)), np.zeros((len(ctx), H, D))
    ref[np.array(ctx) > 0], slack[np.array(ctx) > 0] = ref_live, slack_live
    c["q"] = full
    d = on_device(c)
    out = run(pkv, c, d, scale, cap, slopes)
    assert pkv.get_device_error() == 0
    check(out, c, ref, slack)
    assert (out[np.array(ctx) == 0] == 0).all()
    # the same bits again, in a workspace that starts as NaN
    import torch
    ws = pkv.alloc_grouped_workspace(len(ctx), H, HK, D, B, c["bt"].shape[1])
    ws.fill_(255)
    again = run(pkv, c, d, scale, cap, slopes, workspace=ws)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))


@pytest.mark.parametrize("scale", [0.0, -0.3, 4.0])
def test_scales(pkv, scale):
    """No scale (the mean of the values), a negative one, a steep softmax."""
    c = make_case(np.random.default_rng(3), 6, 2, 64, 16, [1, 1], [50, 700], "f16")
    ref, slack = reference(c, scale, 0.0, None)
    check(run(pkv, c, on_device(c), scale), c, ref, slack)


def test_negative_slopes_favour_far_tokens(pkv):
    c = make_case(np.random.default_rng(4), 4, 1, 128, 16, [1], [900], "bf16")
    slopes = np.array([-0.5, 0.0, 0.25, -3.0], np.float32)
    ref, slack = reference(c, 0.1, 0.0, slopes)
    check(run(pkv, c, on_device(c), 0.1, slopes=slopes), c, ref, slack)


def test_infinite_and_nan_inputs_stay_in_their_sequence(pkv):
    """A NaN key spoils the heads that read it and no other sequence or head."""
    c = make_case(np.random.default_rng(5), 8, 2, 64, 16, [1, 1, 1], [40, 40, 40], "f16")
    ref, slack = reference(c, 0.125, 0.0, None)
    d = on_device(c)
    d["kc"][int(c["bt"][1, 0]), 1, 3, 5] = float("nan")
    out = run(pkv, c, d, 0.125)
    assert out[1, 4:].isnan().all() and out[1, :4].isfinite().all()
    check(out[[0, 2]], c, ref[[0, 2]], slack[[0, 2]])


def test_bad_entries_and_lengths_are_flagged(pkv):
    from paged_kv_cache_05_gb300.pagedkv import DEVERR_BAD_BLOCK, DEVERR_BAD_CONTEXT
    import torch
    rs = np.random.default_rng(6)
    c = make_case(rs, 4, 2, 64, 16, [1, 1, 1], [40, 90, 20], "f16", wild=False)
    ref, slack = reference(c, 0.125, 0.0, None)
    d = on_device(c)
    d["kc"].nan_to_num_(0.0)
    d["vc"].nan_to_num_(0.0)
    d["bt"][1, 2] = c["nb"]
    out = run(pkv, c, d, 0.125)
    assert pkv.get_device_error() == DEVERR_BAD_BLOCK and pkv.get_device_error() == 0
    check(out[[0, 2]], c, ref[[0, 2]], slack[[0, 2]])
    d["bt"].fill_(0)
    d["cl"].copy_(torch.tensor([-3, 1 << 30, 20], dtype=torch.int32))
    out = run(pkv, c, d, 0.125)
    assert pkv.get_device_error() == DEVERR_BAD_CONTEXT
    assert (out[0] == 0).all() and out.isfinite().all()


def test_a_wait_that_runs_out_is_reported(pkv):
    from paged_kv_cache_05_gb300.pagedkv import DEVERR_TIMEOUT
    c = make_case(np.random.default_rng(7), 8, 2, 128, 16, [1] * 8, [3000] * 8, "bf16", wild=False)
    d = on_device(c)
    before = pkv.set_decode_wait_limit(0)
    try:
        run(pkv, c, d, 0.1)
        assert pkv.get_device_error() in (0, DEVERR_TIMEOUT)
    finally:
        pkv.set_decode_wait_limit(before)
    ref, slack = reference(c, 0.1, 0.0, None)
    check(run(pkv, c, d, 0.1), c, ref, slack)
    assert pkv.get_device_error() == 0


def test_captured_replayed_and_on_two_streams(pkv):
    """One captured call, replayed after the lengths and the queries changed; two
    calls on two streams at once, each with its workspace."""
    import torch
    rs = np.random.default_rng(8)
    c = make_case(rs, 16, 4, 128, 16, [1] * 5, [700, 33, 1, 256, 2000], "f16")
    d = on_device(c)
    ws = [pkv.alloc_grouped_workspace(5, 16, 4, 128, 16, c["bt"].shape[1]) for _ in range(2)]
    out = torch.empty_like(d["q"])
    call = lambda o, w, s=None: pkv.paged_attention_decode_grouped(  # noqa: E731
        o, d["q"], d["kc"], d["vc"], d["bt"], d["cl"], 0.09, workspace=w, stream=s)
    call(out, ws[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out, ws[0])
    for k in range(3):
        if k:
            c["ctx"] = np.maximum(c["ctx"] - 7 * k, 0).astype(np.int32)
            d["cl"].copy_(torch.from_numpy(c["ctx"]))
            d["q"].mul_(0.5)
        out.zero_()
        graph.replay()
        want = torch.empty_like(out)
        call(want, ws[1])
        assert torch.equal(out, want)
        graph.replay()
        assert torch.equal(out, want)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.zeros_like(out) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for o, w, s in zip(outs, ws, streams):
            call(o, w, s)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)
    for s in streams:                                    # a workspace of the call's own
        call(outs[0], None, s)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and pkv.get_device_error() == 0


def test_pool_past_32_bit_offsets(pkv):
    """Blocks whose element offsets pass 2^32."""
    import torch
    HK, B, D, H = 8, 16, 128, 16
    nb = (1 << 32) // (HK * B * D) + 50
    kc = torch.zeros((nb, HK, B, D), dtype=torch.float16, device="cuda")
    vc = torch.zeros((nb, HK, B, D), dtype=torch.float16, device="cuda")
    c = make_case(np.random.default_rng(9), H, HK, D, B, [1, 1], [37, 300], "f16", wild=False)
    d = on_device(c)
    far = nb - c["nb"]
    kc[far:], vc[far:] = d["kc"], d["vc"]
    ref, slack = reference(c, 0.09, 0.0, None)
    out = torch.empty_like(d["q"])
    pkv.paged_attention_decode_grouped(out, d["q"], kc, vc, d["bt"] + far, d["cl"], 0.09)
    assert pkv.get_device_error() == 0
    check(out, c, ref, slack)


def test_many_sequences(pkv):
    """More sequences than threads of a block, most of them empty."""
    import torch
    S = 5000
    ctx = [0] * S
    for s in (3, 4, 129, 2500, 4999):
        ctx[s] = 40 + s % 50
    c = make_case(np.random.default_rng(10), 4, 2, 64, 16, [1 if n else 0 for n in ctx], ctx,
                  "bf16")
    ref, slack = reference(c, 0.125, 0.0, None)
    live = np.array(ctx) > 0
    d = on_device(c)
    q = torch.zeros((S, 4, 64), dtype=torch.bfloat16, device="cuda")
    q[torch.from_numpy(live).cuda()] = d["q"]
    d["q"] = q
    out = run(pkv, c, d, 0.125)
    assert pkv.get_device_error() == 0
    check(out[torch.from_numpy(live).cuda()], c, ref, slack)
    assert (out[torch.from_numpy(~live).cuda()] == 0).all()
