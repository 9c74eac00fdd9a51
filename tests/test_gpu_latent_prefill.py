"""Expanded latent attention of ragged prompts and chunks, against the fp64 definition;
rows of no sequence hold NaN."""
import numpy as np
import pytest

from helpers import to_dev
from latent_helpers import check_prefill, prefill_case, run_prefill
from paged_kv_cache_05_gb300 import workloads as W

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_05_gb300 import build
    build.build()
    import paged_kv_cache_05_gb300 as m
    return m


@pytest.mark.parametrize("H,N,new,keys,dtype", [
    (1, 128, [1], [1], "bf16"),
    (2, 64, [1], [200], "f16"),
    (3, 128, [61], [61], "bf16"),
    (2, 128, [128, 127, 129], [128, 127, 129], "f16"),
    (1, 64, [256, 1, 257], [256, 1, 257], "bf16"),
    (5, 64, [3, 0, 70], [3, 0, 70], "f16"),
    (2, 128, [0, 100, 0, 0, 30], [0, 300, 20, 0, 31], "bf16"),
    (2, 64, [130, 7], [700, 7], "f16"),
    (1, 128, [300], [301], "bf16"),
    (16, 128, [5], [513], "f16"),
    (1, 128, [513], [1025], "f16"),
])
def test_shapes(pkv, H, N, new, keys, dtype):
    rs = np.random.RandomState(H + N + sum(keys))
    check_prefill(pkv, prefill_case(rs, H, N, new, keys, dtype), (N + 64) ** -0.5)


@pytest.mark.parametrize("dtype,qtimes", [("f16", 30.0), ("bf16", 30.0), ("bf16", 0.01)])
def test_sharp_and_flat_scores(pkv, dtype, qtimes):
    rs = np.random.RandomState(2)
    check_prefill(pkv, prefill_case(rs, 2, 128, [150], [420], dtype, qtimes), 0.07)


def test_first_row_is_its_value(pkv):
    import torch
    rs = np.random.RandomState(3)
    for dtype in ("f16", "bf16"):
        c = prefill_case(rs, 4, 128, [9, 150], [9, 150], dtype)
        got = run_prefill(pkv, c, 0.07)
        v = to_dev(c["up"], dtype)[..., 128:]
        assert torch.equal(got[0], v[0]) and torch.equal(got[9], v[9])


def test_growing_scores(pkv):
    import torch
    rs = np.random.RandomState(4)
    c = prefill_case(rs, 1, 128, [200], [900], "bf16")
    q, rows = (W.words_to_torch(c[n], "bf16").float() for n in ("q", "rows"))
    q[:200, :, 128] = 20.0
    rows[:900, c["pad"]] = torch.arange(900) / 4
    c["q"], c["rows"] = (W.torch_to_words(x.to(torch.bfloat16)) for x in (q, rows))
    check_prefill(pkv, c, 0.07)


def test_bad_lengths(pkv):
    import torch
    rs = np.random.RandomState(5)
    c = prefill_case(rs, 2, 64, [20, 30, 40], [20, 60, 40], "f16")
    good = run_prefill(pkv, c, 0.07)
    d = {n: to_dev(c[n], "f16") for n in ("q", "up", "rows")}

    def run(qs, ks, mq=40, mk=60):
        out = torch.full((90, 2, 64), 7.0, dtype=torch.float16, device="cuda")
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        pkv.latent_attention_prefill(out, d["q"][:90], d["up"][:120, :, :64], d["rows"][:120, 8:],
                                     d["up"][:120, :, 64:], i32(qs), i32(ks), 0.07, mq, mk)
        return out, pkv.get_device_error()

    out, err = run([0, 20, 50, 90], [0, 20, 80, 120])
    assert err == 0 and torch.equal(out, good)
    for qs, ks, mq, mk, left in (
            ([0, 20, 50, 90], [0, 20, 80, 119], 40, 60, 2),      # fewer keys than rows
            ([0, 20, 50, 91], [0, 20, 80, 120], 41, 60, 2),      # rows past the tensor
            ([0, 20, 50, 90], [0, 20, 80, 130], 40, 60, 2),      # keys past it
            ([0, 20, 50, 90], [0, 20, 80, 120], 30, 60, 2),      # more rows than said
            ([0, 20, 50, 90], [0, 20, 80, 120], 40, 59, 1)):     # more keys than said
        out, err = run(qs, ks, mq, mk)
        assert err == 4
        parts, full = [out[:20], out[20:50], out[50:]], [good[:20], good[20:50], good[50:]]
        for i in range(3):
            assert (parts[i] == 7).all() if i == left else torch.equal(parts[i], full[i])


def test_contiguous_inputs_same_bits_and_streams(pkv):
    import torch
    rs = np.random.RandomState(6)
    c = prefill_case(rs, 3, 128, [70, 300], [400, 300], "bf16")
    want = run_prefill(pkv, c, 0.07)
    d = {n: to_dev(c[n], "bf16") for n in ("q", "up", "rows")}
    k, v, r = (x.contiguous() for x in (d["up"][..., :128], d["up"][..., 128:], d["rows"][:, 8:]))
    qs, ks = torch.from_numpy(c["qs"]).cuda(), torch.from_numpy(c["ks"]).cuda()
    torch.cuda.synchronize()
    outs = [torch.empty(c["q"].shape[0], 3, 128, dtype=torch.bfloat16, device="cuda")
            for _ in range(4)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for i, out in enumerate(outs):
        pkv.latent_attention_prefill(out, d["q"], k, r, v, qs, ks, 0.07, 300, 400,
                                     stream=streams[i % 2])
    torch.cuda.synchronize()
    assert all(torch.equal(out[:c["Tq"]], want) for out in outs)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkv.latent_attention_prefill(outs[0], d["q"], k, r, v, qs, ks, 0.07, 300, 400)
    outs[0].zero_()
    g.replay()
    assert torch.equal(outs[0][:c["Tq"]], want)
    assert pkv.get_device_error() == 0
