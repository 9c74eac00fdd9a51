"""Absorbed latent attention of new tokens, chains and trees over a paged latent cache,
against the fp64 definition; hidden places hold NaN."""
import numpy as np
import pytest

from latent_helpers import check_decode, decode_case, on_device, run_decode

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_05_gb300 import build
    build.build()
    import paged_kv_cache_05_gb300 as m
    return m


@pytest.mark.parametrize("H,R,B,new,ctx,dtype,tree", [
    (16, 512, 16, [1], [1], "bf16", False),
    (1, 256, 8, [1], [5], "f16", False),
    (128, 512, 64, [1], [64], "bf16", False),
    (16, 512, 16, [1], [129], "f16", False),
    (16, 512, 8, [1, 1, 1], [127, 128, 300], "bf16", False),
    (3, 256, 32, [1] * 5, [1, 31, 33, 255, 700], "bf16", False),
    (128, 512, 16, [1, 1], [17, 611], "f16", False),
    (129, 256, 16, [1], [200], "bf16", False),
    (65, 512, 32, [1, 1], [140, 3], "f16", False),
    (200, 256, 64, [2, 1], [259, 70], "f16", False),
    (16, 512, 16, [7, 1, 0, 13], [7, 200, 50, 333], "bf16", False),
    (20, 256, 32, [13, 1, 5], [77, 140, 5], "f16", True),
    (8, 512, 8, [64], [200], "bf16", True),
    (32, 256, 16, [33, 64, 2], [300, 64, 129], "f16", True),
    (5, 512, 64, [40], [100], "f16", False),
    (16, 256, 16, [150], [400], "bf16", False),
    (16, 512, 16, [1] * 90, [1 + 7 * i for i in range(90)], "bf16", False),
])
def test_shapes(pkv, H, R, B, new, ctx, dtype, tree):
    rs = np.random.RandomState(H + R + sum(ctx))
    c = decode_case(rs, H, R, B, new, ctx, dtype, tree)
    check_decode(pkv, c, 192 ** -0.5)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_long_and_short(pkv, dtype):
    rs = np.random.RandomState(3)
    c = decode_case(rs, 16, 512, 16, [1, 1, 2], [9000, 3, 1100], dtype)
    check_decode(pkv, c, 192 ** -0.5)


def test_empty_sequences_are_zero(pkv):
    rs = np.random.RandomState(4)
    c = decode_case(rs, 16, 512, 16, [1, 1, 1], [0, 40, 0], "bf16")
    got = check_decode(pkv, c, 0.07)
    assert (got[0] == 0).all() and (got[2] == 0).all()


def test_rows_that_see_nothing_are_zero(pkv):
    """A tree at the head of a sequence, one row of which has no bit set."""
    rs = np.random.RandomState(5)
    c = decode_case(rs, 20, 256, 16, [5, 3], [5, 60], "f16", tree=True)
    c["tree"][2] = 0
    c["tree"][1] = 1 << 40 | 1 << 63               # bits past the rows are ignored
    got = check_decode(pkv, c, 0.07)
    assert (got[2] == 0).all() and (got[1] == 0).all() and not (got[6] == 0).any()


def test_one_token_gives_its_row(pkv):
    """A row that sees one token is that token's latent part, bit for bit."""
    import torch
    rs = np.random.RandomState(6)
    for dtype in ("f16", "bf16"):
        c = decode_case(rs, 70, 512, 16, [1], [1], dtype)
        d = on_device(c)
        got = run_decode(pkv, c, 0.3, d)
        want = d["cache"][c["bt"][0, 0], 0, :512].expand(70, 512)
        assert torch.equal(got[0], want)


@pytest.mark.parametrize("dtype,qtimes", [("f16", 30.0), ("bf16", 30.0), ("f16", 0.01)])
def test_sharp_and_flat_scores(pkv, dtype, qtimes):
    """Softmaxes with one large weight, which the running max has to find late as well as
    early, and nearly equal ones."""
    rs = np.random.RandomState(7)
    c = decode_case(rs, 32, 256, 16, [1, 3], [640, 300], dtype, qtimes=qtimes)
    check_decode(pkv, c, 0.07)


def test_growing_scores(pkv):
    """Keys whose scores grow along the context by far more than a weight's range: the
    accumulated output is rescaled again and again."""
    from paged_kv_cache_05_gb300 import workloads as W
    import torch
    rs = np.random.RandomState(8)
    c = decode_case(rs, 16, 512, 16, [1], [900], "bf16")
    cache = W.words_to_torch(c["cache"], "bf16").float()
    q = W.words_to_torch(c["q"], "bf16").float()
    q[..., 512] = 20.0
    for t in range(900):
        cache[c["bt"][0, t // 16], t % 16, 512] = float(t) / 4
    c["q"], c["cache"] = (W.torch_to_words(x.to(torch.bfloat16)) for x in (q, cache))
    check_decode(pkv, c, 0.07)


def test_many_small_weights_beside_a_large_one(pkv):
    """fp16 weights of 2^-20 of the largest, twenty thousand of them: their sum is a fiftieth
    of the result."""
    import torch
    n, R, B = 20000, 256, 64
    nb = -(-n // B)
    cache = torch.zeros(nb * B, R + 64, dtype=torch.float16, device="cuda")
    cache[0, R] = 1.0                              # score 20 log2 units above the others
    cache[1:n, 0] = 1.0
    q = torch.zeros(1, 16, R + 64, dtype=torch.float16, device="cuda")
    q[..., R] = 20.0
    out = torch.empty(1, 16, R, dtype=torch.float16, device="cuda")
    pkv.latent_attention_decode(out, q, cache.view(nb, B, R + 64),
                                torch.arange(nb, dtype=torch.int32, device="cuda")[None],
                                torch.tensor([n], dtype=torch.int32, device="cuda"),
                                float(np.log(2.0)))
    want = (n - 1) * 2.0 ** -20 / (1 + (n - 1) * 2.0 ** -20)
    # the weights' rounding (2^-11) twice, the output's once
    assert (out[0, :, 0].double() - want).abs().max().item() <= 3 * 2.0 ** -11 * want


def test_bad_lengths_and_blocks(pkv):
    import torch
    rs = np.random.RandomState(9)
    c = decode_case(rs, 16, 256, 16, [1] * 4, [20, 40, 33, 50], "f16")
    good = run_decode(pkv, c, 0.07)
    assert pkv.get_device_error() == 0
    d = on_device(c)
    d["cl"][1] = -3
    d["cl"][3] = 16 * c["bt"].shape[1] + 1
    got = run_decode(pkv, c, 0.07, d)
    assert pkv.get_device_error() == 4
    assert torch.equal(got[[0, 2]], good[[0, 2]]) and (got[[1, 3]] == 7).all()
    d = on_device(c)
    d["bt"][2, 1] = -1                             # tokens 16 .. 31 are left out
    got = run_decode(pkv, c, 0.07, d)
    assert pkv.get_device_error() == 1
    assert torch.equal(got[[0, 1, 3]], good[[0, 1, 3]])
    k = d["cache"][c["bt"][2, [0, 2]]].reshape(-1, 320)[:17].double()
    want = torch.softmax(0.07 * d["q"][2].double() @ k.T, -1) @ k[:, :256]
    assert (got[2].double() - want).abs().max() <= 4e-3
    # more rows than the caller said, rows past the tensor
    c = decode_case(rs, 16, 256, 16, [1, 3, 1], [20, 40, 33], "f16")
    d = on_device(c)
    out = torch.full((5, 16, 256), 7.0, dtype=torch.float16, device="cuda")
    args = (d["q"], d["cache"], d["bt"], d["cl"], 0.07)
    pkv.latent_attention_decode(out, *args, query_start=d["qs"], max_query_len=2)
    assert pkv.get_device_error() == 4
    assert (out[1:4] == 7).all() and not (out[0] == 7).all() and not (out[4] == 7).all()
    d["qs"][3] = 9
    pkv.latent_attention_decode(out, *args, query_start=d["qs"], max_query_len=8)
    assert pkv.get_device_error() == 4


def test_without_query_start(pkv):
    import torch
    rs = np.random.RandomState(10)
    c = decode_case(rs, 16, 512, 32, [1] * 3, [20, 400, 33], "bf16")
    d = on_device(c)
    out = torch.empty(3, 16, 512, dtype=torch.bfloat16, device="cuda")
    pkv.latent_attention_decode(out, d["q"], d["cache"], d["bt"], d["cl"], 0.07)
    assert torch.equal(out, run_decode(pkv, c, 0.07, d))


def test_same_bits_from_call_to_call(pkv):
    import torch
    rs = np.random.RandomState(11)
    c = decode_case(rs, 16, 512, 16, [1, 5, 1], [2000, 700, 90], "bf16")
    d = on_device(c)
    first = run_decode(pkv, c, 0.07, d)
    for _ in range(5):
        assert torch.equal(first, run_decode(pkv, c, 0.07, d))


def test_two_calls_at_once_and_graph(pkv):
    """Calls on two streams with workspaces of their own, and a captured call replayed on
    new inputs."""
    import torch
    rs = np.random.RandomState(12)
    cases = [decode_case(rs, 16, 512, 16, [1, 1], [n, 200], "bf16") for n in (1500, 900)]
    dev = [on_device(c) for c in cases]
    want = [run_decode(pkv, c, 0.07, d) for c, d in zip(cases, dev)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(10):
        got = []
        for c, d, st in zip(cases, dev, streams):
            with torch.cuda.stream(st):
                got.append(run_decode(pkv, c, 0.07, d))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    c, d = cases[0], dev[0]
    ws = pkv.alloc_latent_workspace(2, 16, 512)
    out = torch.empty_like(want[0])
    args = dict(query_start=d["qs"], max_query_len=1, workspace=ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkv.latent_attention_decode(out, d["q"], d["cache"], d["bt"], d["cl"], 0.07, **args)
    g.replay()
    assert torch.equal(out, want[0])
    d["q"].mul_(0.5)
    d["cl"][0] = 700
    g.replay()
    fresh = torch.empty_like(out)
    pkv.latent_attention_decode(fresh, d["q"], d["cache"], d["bt"], d["cl"], 0.07, **args)
    assert torch.equal(out, fresh) and not torch.equal(out, want[0])
    assert pkv.get_device_error() == 0
