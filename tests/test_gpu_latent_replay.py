"""Latent attention captured once and replayed on other lengths, trees and padded places; long
calls side by side on two streams; heads of 64 with several items a head."""
import numpy as np
import pytest

from helpers import to_dev
from latent_helpers import (check_decode, check_prefill, decode_case, on_device, prefill_case,
                            run_prefill, to_i64)
from paged_kv_cache_05_gb300 import workloads as W

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_05_gb300 import build
    build.build()
    import paged_kv_cache_05_gb300 as m
    return m


def prompt_args(c):
    import torch
    d = {n: to_dev(c[n], c["dtype"]) for n in ("q", "up", "rows")}
    return ([d["q"], d["up"][..., :c["N"]], d["rows"][:, c["pad"]:], d["up"][..., c["N"]:],
             torch.from_numpy(c["qs"]).cuda(), torch.from_numpy(c["ks"]).cuda()])


@pytest.mark.parametrize("N,dtype", [(128, "bf16"), (64, "f16")])
def test_captured_prompts_of_other_lengths(pkv, N, dtype):
    """A captured call over four places, replayed when two of them are empty, then when one
    sequence fills all rows; each replay gives the bits of a fresh call and leaves the rows of
    no sequence alone."""
    import torch
    rs = np.random.RandomState(21)
    new, keys = [130, 1, 300, 89], [700, 90, 300, 910]
    c = prefill_case(rs, 3, N, new, keys, dtype)
    args = prompt_args(c)
    qs, ks = args[4:]
    out = torch.full((c["q"].shape[0], 3, N), 7.0, dtype=W.torch_dtype(dtype), device="cuda")
    mq, mk = sum(new), sum(keys)
    ws = torch.empty(pkv.latent_prefill_workspace_size(N, mq, mk), dtype=torch.uint8, device="cuda")

    def call(o):
        return pkv.latent_attention_prefill(o, *args, 0.1, mq, mk, workspace=ws)

    call(out)
    assert torch.equal(out[:c["Tq"]], run_prefill(pkv, c, 0.1))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(out)
    for starts, ends in (([0, 130, 130, 330, 330], [0, 500, 500, 900, 900]),
                         ([0, 0, 520, 520, 520], [0, 0, 2000, 2000, 2000]),
                         ([0, 0, 0, 0, 0], [0, 0, 0, 0, 0]),
                         (c["qs"], c["ks"])):
        qs.copy_(torch.tensor(np.array(starts), dtype=torch.int32))
        ks.copy_(torch.tensor(np.array(ends), dtype=torch.int32))
        out.fill_(7.0)
        g.replay()
        fresh = call(torch.full_like(out, 7.0))
        n = int(starts[-1])
        assert torch.equal(out, fresh) and (out[n:] == 7.0).all()
        assert torch.isfinite(out[:n]).all()
    assert pkv.get_device_error() == 0


def test_long_prompts_on_two_streams(pkv):
    """Calls whose items are cut, with memory of their own, side by side."""
    import torch
    rs = np.random.RandomState(22)
    cases = [prefill_case(rs, 2, N, [n], [n + 600], "bf16") for N, n in ((128, 700), (64, 530))]
    want = [run_prefill(pkv, c, 0.1) for c in cases]
    args = [prompt_args(c) for c in cases]
    outs = [torch.empty(c["q"].shape[0], 2, c["N"], dtype=torch.bfloat16, device="cuda")
            for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(10):
        for c, a, o, st in zip(cases, args, outs, streams):
            with torch.cuda.stream(st):
                pkv.latent_attention_prefill(o, *a, 0.1, c["new"][0], c["keys"][0])
    torch.cuda.synchronize()
    for c, o, w in zip(cases, outs, want):
        assert torch.equal(o[:c["Tq"]], w)
    assert pkv.get_device_error() == 0


@pytest.mark.parametrize("dtype,qtimes", [("f16", 1.0), ("bf16", 30.0)])
def test_narrow_heads_of_several_items(pkv, dtype, qtimes):
    rs = np.random.RandomState(23)
    c = prefill_case(rs, 3, 64, [700, 40, 1030], [1500, 40, 1100], dtype, qtimes)
    check_prefill(pkv, c, 64 ** -0.5)


def test_narrow_heads_growing_scores(pkv):
    import torch
    rs = np.random.RandomState(24)
    c = prefill_case(rs, 1, 64, [300], [900], "bf16")
    q, rows = (W.words_to_torch(c[n], "bf16").float() for n in ("q", "rows"))
    q[:300, :, 64] = 20.0
    rows[:900, c["pad"]] = torch.arange(900) / 4
    c["q"], c["rows"] = (W.torch_to_words(x.to(torch.bfloat16)) for x in (q, rows))
    check_prefill(pkv, c, 0.07)


def test_captured_trees(pkv):
    """A captured call over four places replayed with other trees, with a place that has
    become empty (its rows 0) and with shorter sequences."""
    import torch
    rs = np.random.RandomState(25)
    new, ctx = [13, 1, 7, 13], [1500, 40, 129, 13]
    c = decode_case(rs, 20, 256, 16, new, ctx, "f16", tree=True)
    check_decode(pkv, c, 0.08)
    d = on_device(c)
    ws = pkv.alloc_latent_workspace(4, 20, 256, 13)
    out = torch.full((sum(new), 20, 256), 7.0, dtype=torch.float16, device="cuda")

    def call(o):
        return pkv.latent_attention_decode(o, d["q"], d["cache"], d["bt"], d["cl"], 0.08,
                                           query_start=d["qs"], max_query_len=13,
                                           ancestors=d["tree"], workspace=ws)

    call(out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(out)
    other = decode_case(rs, 20, 256, 16, new, ctx, "f16", tree=True)["tree"]
    for tree, lens, empty in ((other, ctx, None), (other, [900, 40, 0, 13], 2),
                              (c["tree"], [13, 1, 7, 0], 3), (c["tree"], ctx, None)):
        d["tree"].copy_(torch.from_numpy(to_i64(tree)))
        d["cl"].copy_(torch.tensor(lens, dtype=torch.int32))
        out.fill_(7.0)
        g.replay()
        assert torch.equal(out, call(torch.full_like(out, 7.0)))
        assert torch.isfinite(out).all()
        for s in range(4):
            rows = out[int(c["qs"][s]):int(c["qs"][s + 1])]
            assert bool((rows == 0).all()) == (s == empty)
    assert pkv.get_device_error() == 0
