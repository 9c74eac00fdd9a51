"""The prompt phase of few new tokens over long caches with shared K/V heads:
items cut along the keys, their parts joined, against the fp64 definition.

Bound: test_gpu_prefill_grouped's, and the join's own: a part's weights and sums
are relative to its own running max and scaled by a power of at most 1, so what
they round to fewer bits weighs no more than there; the scaling (2^-22, the fast
exponential), and fp32 sums of at most 32 parts (32 steps of 2^-24) add at most
2^-18 of sum p |v| / sum p, a quarter of the 2^-16 of it in the bound.
"""
import math

import numpy as np
import pytest

from grouped_helpers import check, make_case, on_device
from test_gpu_prefill_grouped import alibi, bounded, pkv, run  # noqa: F401

pytestmark = pytest.mark.gpu


def space(pkv, c, d, most=None):
    """A workspace full of NaN, 64 bytes longer than it has to be."""
    import torch
    n = pkv.prefill_grouped_workspace_size(len(c["ctx"]), c["H"], c["HK"], c["D"], c["B"],
                                           c["bt"].shape[1], most or max(max(c["new"]), 1))
    assert n > 0
    return torch.full((n + 64,), 0xFF, dtype=torch.uint8, device="cuda"), n


CASES = [
    # H, HK, D, B, dtype, new, past, window, softcap, biased
    (8, 2, 128, 16, "bf16", [1, 4, 8], 3000, 0, 0.0, False),
    (8, 8, 64, 8, "f16", [5], 4500, 0, 0.0, False),
    (7, 1, 64, 32, "bf16", [3, 0, 40], 2500, 0, 30.0, False),
    (13, 1, 128, 64, "f16", [9, 1], 4000, 0, 0.0, True),
    (6, 2, 128, 16, "bf16", [300, 2], 2700, 1500, 0.0, False),
    (4, 1, 64, 16, "f16", [129], 3333, 1000, 20.0, True),
    (3, 1, 128, 8, "bf16", [257, 1], 1500, 0, 0.0, True),
    (16, 1, 128, 16, "bf16", [2] * 6 + [0, 1], 2000, 0, 0.0, False),
    (1, 1, 128, 16, "f16", [700], 9000, 0, 0.0, False),
    (1, 1, 64, 64, "bf16", [1], 20001, 0, 8.0, False),
    (67, 1, 64, 16, "f16", [2], 1300, 0, 0.0, False),
    (2, 1, 128, 16, "f16", [4], 1024, 5, 0.0, False),
    (40, 8, 64, 8, "bf16", [2, 60, 101, 33], 2600, 0, 0.0, True),
    (12, 2, 128, 32, "f16", [20, 1, 17], 1200, 900, 0.0, False),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "%dx%d-D%d-B%d-%s-new%d-past%d-w%d-c%g-%d" % (
    c[0], c[1], c[2], c[3], c[4], max(c[5]), c[6], c[7], c[8], c[9]))
def test_against_fp64(pkv, case):  # noqa: F811
    import torch
    H, HK, D, B, dtype, new, past, window, cap, biased = case
    rs = np.random.default_rng(H * 100 + D + B + past + window)
    ctx = [n + past - 131 * i if n else 0 for i, n in enumerate(new)]
    c = make_case(rs, H, HK, D, B, new, ctx, dtype, window, 6.0 if cap else 1.0)
    slopes = alibi(H) if biased else None
    scale = 1 / math.sqrt(D)
    ref, slack = bounded(c, scale, cap, slopes)
    d = on_device(c)
    ws, n = space(pkv, c, d)
    out = run(pkv, c, d, scale, cap, slopes, workspace=ws[:n])
    assert pkv.get_device_error() == 0
    check(out, c, ref, slack * 1.25)
    assert (ws[n:] == 0xFF).all()
    # the same bits with the parts in the workspace again, and in one of the call's own
    again = run(pkv, c, d, scale, cap, slopes, workspace=ws[:n])
    own = run(pkv, c, d, scale, cap, slopes)
    for o in (again, own):
        assert torch.equal(o.view(torch.int16), out.view(torch.int16))


def test_a_batch_that_is_not_cut_after_one_that_was(pkv):  # noqa: F811
    """The capacity of the tables allows a cut, the lengths do not ask for one."""
    rs = np.random.default_rng(5)
    long = make_case(rs, 8, 2, 64, 16, [3, 2], [2500, 1800], "bf16")
    d = on_device(long)
    ws, n = space(pkv, long, d)
    scale = 0.125
    ref, slack = bounded(long, scale, 0.0, None)
    check(run(pkv, long, d, scale, workspace=ws[:n]), long, ref, slack * 1.25)
    short = make_case(rs, 8, 2, 64, 16, [3, 2], [9, 2], "bf16")
    short["bt"] = np.concatenate([short["bt"], np.full((2, 160), -1, np.int32)], 1)
    ref, slack = bounded(short, scale, 0.0, None)
    check(run(pkv, short, on_device(short), scale, workspace=ws[:n]), short, ref, slack)
    assert pkv.get_device_error() == 0


def test_rows_of_one_head_need_the_others_not(pkv):  # noqa: F811
    """A query tile holds rows of several heads: a NaN query spoils its own only."""
    import torch
    c = make_case(np.random.default_rng(15), 8, 2, 128, 16, [5, 3], [2100, 900], "f16")
    d = on_device(c)
    ref, slack = bounded(c, 0.09, 0.0, None)
    d["q"][2, 3] = float("nan")
    out = run(pkv, c, d, 0.09)
    assert out[2, 3].isnan().all()
    out[2, 3] = torch.from_numpy(ref[2, 3]).to(out)
    check(out, c, ref, slack * 1.25)


def test_a_bad_block_is_flagged(pkv):  # noqa: F811
    from paged_kv_cache_05_gb300.pagedkv import DEVERR_BAD_BLOCK
    c = make_case(np.random.default_rng(6), 4, 2, 64, 16, [4, 9], [1500, 2000], "f16", wild=False)
    ref, slack = bounded(c, 0.125, 0.0, None)
    d = on_device(c)
    d["kc"].nan_to_num_(0.0)
    d["vc"].nan_to_num_(0.0)
    d["bt"][1, 70] = 1 << 30
    out = run(pkv, c, d, 0.125)
    assert pkv.get_device_error() == DEVERR_BAD_BLOCK and pkv.get_device_error() == 0
    check(out[:4], c, ref[:4], slack[:4] * 1.25)


def test_captured_on_two_streams(pkv):  # noqa: F811
    """Two captured calls, each with its own workspace, replayed side by side
    while the inputs change."""
    import torch
    c = make_case(np.random.default_rng(8), 8, 2, 128, 16, [4, 33], [3000, 1700], "bf16", 2000,
                  wild=False)
    d = on_device(c)
    most = 33
    q = [d["q"].clone(), d["q"] * 0.5]
    outs = [torch.empty_like(x) for x in q]
    spaces = [space(pkv, c, d)[0] for _ in q]
    streams = [torch.cuda.Stream() for _ in q]

    def call(out, x, ws, stream=None):
        pkv.paged_attention_prefill_grouped(out, x, d["kc"], d["vc"], d["bt"], d["cl"], d["qs"],
                                            0.09, most, window=2000, workspace=ws, stream=stream)

    graphs = []
    for out, x, ws in zip(outs, q, spaces):
        call(out, x, ws)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(out, x, ws)
        graphs.append(graph)
    for k in range(3):
        for x, out in zip(q, outs):
            x.mul_(1.25)
            out.zero_()
        torch.cuda.synchronize()
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                for _ in range(4):
                    graph.replay()
        torch.cuda.synchronize()
        for x, out in zip(q, outs):
            want = torch.empty_like(out)
            call(want, x, None)
            torch.cuda.synchronize()
            assert torch.equal(out.view(torch.int16), want.view(torch.int16))
    assert pkv.get_device_error() == 0


@pytest.mark.parametrize("S,H,HK,new", [(40, 16, 1, 90), (5, 24, 3, 700), (2, 7, 7, 1500)])
def test_tiles_of_fewer_heads(pkv, S, H, HK, new):  # noqa: F811
    """Many items: the tiles take fewer heads each; odd numbers of groups."""
    news = [max(new - 37 * i, 1) for i in range(S)]
    c = make_case(np.random.default_rng(S), H, HK, 64, 16, news, [n + 50 for n in news], "bf16", 300)
    ref, slack = bounded(c, 0.125, 0.0, None)
    check(run(pkv, c, on_device(c), 0.125), c, ref, slack)
    assert pkv.get_device_error() == 0


PAIRS = [
    # items of two tiles: more tiles than SMs
    (16, 4, 128, 16, "bf16", [200, 131, 64, 257, 90], 300, 100, 20.0, True),
    (24, 24, 64, 32, "f16", [300, 290, 129, 257], 200, 129, 0.0, False),
    (32, 8, 64, 8, "bf16", [300, 1, 255, 170], 77, 0, 0.0, True),
    (40, 8, 128, 64, "f16", [260, 130, 77], 0, 64, 30.0, False),
]


@pytest.mark.parametrize("case", PAIRS, ids=lambda c: "%dx%d-D%d-B%d-%s-new%d-past%d-w%d-c%g-%d" % (
    c[0], c[1], c[2], c[3], c[4], max(c[5]), c[6], c[7], c[8], c[9]))
def test_items_of_two_tiles(pkv, case):  # noqa: F811
    H, HK, D, B, dtype, new, past, window, cap, biased = case
    rs = np.random.default_rng(H + D + B + past + window)
    c = make_case(rs, H, HK, D, B, new, [n + max(past - 31 * i, 0) for i, n in enumerate(new)],
                  dtype, window, 6.0 if cap else 1.0)
    slopes = alibi(H) if biased else None
    scale = 1 / math.sqrt(D)
    ref, slack = bounded(c, scale, cap, slopes)
    check(run(pkv, c, on_device(c), scale, cap, slopes), c, ref, slack)
    assert pkv.get_device_error() == 0


@pytest.mark.parametrize("new,past", [([3, 6], 2000), ([40, 70], 0), ([200, 190, 180, 170], 0)])
def test_rows_behind_the_last_sequence(pkv, new, past):  # noqa: F811
    """A padded batch: q and out have more rows than the sequences."""
    import torch
    c = make_case(np.random.default_rng(21), 16, 4, 64, 16, new, [n + past for n in new], "bf16")
    ref, slack = bounded(c, 0.125, 0.0, None)
    d = on_device(c)
    rows = sum(new)
    q = torch.full((rows + 70, 16, 64), float("nan"), dtype=d["q"].dtype, device="cuda")
    q[:rows] = d["q"]
    out = torch.full_like(q, 7.0)
    pkv.paged_attention_prefill_grouped(out, q, d["kc"], d["vc"], d["bt"], d["cl"], d["qs"], 0.125,
                                        max(new))
    assert pkv.get_device_error() == 0
    assert (out[rows:] == 7.0).all()
    check(out[:rows], c, ref, slack * 1.25)


def test_a_call_of_its_own_workspace_on_another_stream(pkv):  # noqa: F811
    """The workspace that a call takes is not given to others before it is done."""
    import torch
    c = make_case(np.random.default_rng(23), 8, 2, 128, 16, [6, 9], [2600, 1900], "f16", wild=False)
    d = on_device(c)
    ref, slack = bounded(c, 0.09, 0.0, None)
    n = space(pkv, c, d)[1]
    side = torch.cuda.Stream()
    outs = [torch.empty_like(d["q"]) for _ in range(6)]
    torch.cuda.synchronize()
    for out in outs:
        pkv.paged_attention_prefill_grouped(out, d["q"], d["kc"], d["vc"], d["bt"], d["cl"], d["qs"],
                                            0.09, 9, stream=side)
        torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    assert pkv.get_device_error() == 0
    for out in outs:
        check(out, c, ref, slack * 1.25)
