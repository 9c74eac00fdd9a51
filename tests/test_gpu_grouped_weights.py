"""Many small weights beside a large one: what they add up to is not lost.

Token 0 has the score z0, all others 0, and its value is 0: with w = 2^-z0' (z0' =
z0 in log2 units) the output is w sum V / (1 + (n - 1) w), nothing but small
weights.  Bound, relative to that output: the score's fp32 error (2^-20 of the
48 + 26 that grouped_helpers counts, twice); the products with V add 16 tokens at a
time and lose up to a whole step, 2^-23, each: n 2^-27; the sum of weights loses, in
a thread that holds a quarter of the tokens and token 0, at most each of them,
2^-25: n 2^-27 again; the weights' own error, at most `quantum` of the largest
weight or 2^-12 of themselves; and the output's rounding, half a step.
"""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

Z0 = 25.2                  # log2 units: alone, such a weight is below fp16's half step 2^-25


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_05_gb300 import build
    build.build()
    import paged_kv_cache_05_gb300 as m
    return m


def pool(n, HK, D, B, dtype, seed):
    """One sequence's n tokens: K zero but for token 0's first element, V in
    [0.5, 1.5) but for token 0's, which is 0; tables in a shuffled order."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    nb = -(-n // B)
    k = torch.zeros((nb * B, HK, D), device="cuda")
    v = torch.rand((nb * B, HK, D), generator=g, device="cuda") + 0.5
    k[0, :, 0] = 1.0
    v[0] = 0.0
    v[n:] = float("nan")
    table = torch.randperm(nb, generator=g, device="cuda").to(torch.int32)
    kc, vc = (torch.empty((nb, HK, B, D), dtype=dtype, device="cuda") for _ in range(2))
    for pages, rows in ((kc, k), (vc, v)):
        pages[table.long()] = rows.to(dtype).view(nb, B, HK, D).transpose(1, 2)
    return kc, vc, table[None], v[:n].to(dtype).double()


def expected(v, n, cap):
    """[HK, D], and the small weights relative to the largest."""
    s = Z0 * math.log(2.0)
    z = cap * math.tanh(s / cap) if cap else s
    w = math.exp(-z)
    return v[:n].sum(0) * w / (1 + (n - 1) * w), w


def check(out, want, w, quantum, n):
    """out [rows, H, D] of heads that share want [HK, D]'s heads."""
    import torch
    rel = 2 * 2.0 ** -20 * 74 + n * 2.0 ** -26 + max(quantum / w, 2.0 ** -12)
    half = torch.finfo(out.dtype).eps / 2
    G = out.shape[1] // want.shape[0]
    want = want.repeat_interleave(G, 0)[None]
    err = ((out.double() - want).abs() / want).max().item()
    assert err <= rel + half * (1 + rel), (err, rel, half)


@pytest.mark.parametrize("S,H,HK,cap", [(64, 32, 16, 0.0), (256, 32, 2, 0.0), (64, 48, 16, 40.0)])
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_decode(pkv, S, H, HK, cap, dtype):
    """So many rows that a warp keeps thousands of tokens beside token 0."""
    import torch
    dtype = getattr(torch, dtype)
    n, D, B = 32768, 64, 64
    kc, vc, table, v = pool(n, HK, D, B, dtype, 3)
    q = torch.zeros((S, H, D), dtype=dtype, device="cuda")
    q[:, :, 0] = 1.0
    out = torch.empty_like(q)
    ctx = torch.full((S,), n, dtype=torch.int32, device="cuda")
    pkv.paged_attention_decode_grouped(out, q, kc, vc, table.repeat(S, 1), ctx,
                                       Z0 * math.log(2.0), softcap=cap)
    assert pkv.get_device_error() == 0
    want, w = expected(v, n, cap)
    check(out, want, w, 2.0 ** -36 if dtype == torch.float16 else 2.0 ** -60, n)


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("cap,biased", [(0.0, False), (40.0, False), (0.0, True), (40.0, True)])
@pytest.mark.parametrize("H,HK,D,cut", [(4, 1, 64, False), (2, 2, 128, False), (8, 2, 128, True)])
def test_prompts(pkv, H, HK, D, cut, cap, biased, dtype):
    import torch
    dtype = getattr(torch, dtype)
    n, m, B = 40000, 3, 64
    kc, vc, table, v = pool(n, HK, D, B, dtype, 4)
    q = torch.zeros((m, H, D), dtype=dtype, device="cuda")
    q[:, :, 0] = 1.0
    out = torch.empty_like(q)
    size = pkv.prefill_grouped_workspace_size(1, H, HK, D, B, table.shape[1], m)
    assert size > 0
    space = torch.empty(size if cut else 0, dtype=torch.uint8, device="cuda")
    t = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    pkv.paged_attention_prefill_grouped(
        out, q, kc, vc, table.contiguous(), t(n), t(0, m), Z0 * math.log(2.0), m, softcap=cap,
        slopes=torch.zeros(H, device="cuda") if biased else None, workspace=space)
    assert pkv.get_device_error() == 0
    for i in range(m):
        want, w = expected(v, n - m + 1 + i, cap)
        check(out[i:i + 1], want, w, 2.0 ** -34 if dtype == torch.float16 else 2.0 ** -60, n)
