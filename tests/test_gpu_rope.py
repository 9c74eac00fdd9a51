"""Norm, rotation and cache write in one pass, against the fp64 definition.

Bound per element, with (a, b) the normed pair it comes from (for an element
that is not turned, a is itself and b is 0): fp32 work is off by at most 24
units of 2^-24 of rope_scale (|a| + |b|) -- the norm's factor 12 (a sum of at
most 128 squares in a tree of 8 + 4 steps, halved by the root, rsqrt 2, two
products), the angle 3.2 (half a turn rounded to 24 bits), sine and cosine 1
each way, the scale 1, two products and a sum 3 -- plus |angle| 2^-51 for the
frequency's own 53 bits here and in the fixed-point form; the result is then
rounded once, half a step of its type (2^-25 at least for fp16's subnormals).
"""
import math

import numpy as np
import pytest

from helpers import to_dev, words
from oracle.grouped import norm_rope
from paged_kv_cache_05_gb300 import workloads as W

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_05_gb300 import build
    build.build()
    import paged_kv_cache_05_gb300 as m
    return m


def f64(w, dtype):
    return W.words_to_torch(w, dtype).double().numpy()


def bound(x, ref, positions, f, weight, eps, rope_scale, interleaved, dtype):
    """The bound above for the rows x, element by element."""
    import torch
    y = norm_rope(x, positions, [], weight, eps)
    pair = np.abs(y)
    angle = np.zeros_like(y)
    n = len(f)
    for i in range(n):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
        s = np.abs(y[..., a]) + np.abs(y[..., b])
        pair[..., a] = pair[..., b] = s * abs(rope_scale)
        angle[..., a] = angle[..., b] = np.abs(np.asarray(positions, np.float64) * f[i])[:, None]
    fp32 = pair * (24 * 2.0 ** -24 + angle * 2.0 ** -51)
    half = torch.finfo(W.torch_dtype(dtype)).eps / 2
    return fp32 + half * (np.abs(ref) + fp32) + (2.0 ** -25 if dtype == "f16" else 0.0)


def check(got, x, positions, f, weight, eps, rope_scale, interleaved, dtype, what):
    ref = norm_rope(x, positions, f, weight, eps, rope_scale, interleaved)
    g = got.double().cpu().numpy()
    err = np.abs(g - ref)
    ok = err <= bound(x, ref, positions, f, weight, eps, rope_scale, interleaved, dtype)
    assert ok.all(), "%s: %d of %d off, worst %g" % (what, (~ok).sum(), ok.size, err.max())


CASES = [
    # T, H, HK, D, rot, B, dtype, norm, interleaved, far
    (1, 32, 8, 128, 128, 16, "bf16", "qk", False, 131072),
    (1, 1, 1, 64, 64, 8, "f16", "", True, 100),
    (3, 5, 3, 64, 24, 32, "f16", "q", False, 2 ** 31 - 1),
    (7, 7, 1, 128, 8, 64, "bf16", "k", True, 2 ** 31 - 1),
    (33, 71, 1, 64, 64, 16, "bf16", "qk", True, 4096),
    (50, 40, 8, 128, 96, 16, "f16", "qk", False, 32768),
    (64, 6, 6, 128, 0, 8, "bf16", "qk", False, 77),
    (129, 9, 3, 64, 40, 16, "f16", "", False, 1000000),
    (2500, 4, 2, 128, 128, 16, "bf16", "qk", False, 131072),
]


def make(case, seed, joint):
    T, H, HK, D, rot, B, dtype, norm, inter, far = case
    rs = np.random.default_rng(seed)
    nb = -(-T // B) + 2
    width = (H + 2 * HK) * D + (24 if joint else 0)
    qkv = words((T, width), dtype, rs)
    c = dict(qkv=qkv, q=qkv[:, :H * D].reshape(T, H, D),
             k=qkv[:, H * D:(H + HK) * D].reshape(T, HK, D),
             v=qkv[:, (H + HK) * D:(H + 2 * HK) * D].reshape(T, HK, D),
             kc=words((nb, HK, B, D), dtype, rs), vc=words((nb, HK, B, D), dtype, rs),
             slots=rs.permutation(nb * B)[:T].astype(np.int64),
             pos=rs.integers(0, far, size=T).astype(np.int32),
             f=10000.0 ** (-np.arange(0, rot, 2) / max(rot, 1)),
             qw=(1 + 0.3 * rs.standard_normal(D)).astype(np.float32) if "q" in norm else None,
             kw=(1 + 0.3 * rs.standard_normal(D)).astype(np.float32) if "k" in norm else None)
    c["pos"][0] = far
    if T > 1:
        c["pos"][-1] = 0
    return c


@pytest.mark.parametrize("case", CASES, ids=lambda c: "T%d-%dx%d-D%d-r%d-%s" % (
    c[0], c[1], c[2], c[3], c[4], c[6]))
@pytest.mark.parametrize("joint", [False, True])
def test_against_fp64(pkv, case, joint):
    """Queries, the key pool and the value pool, the rest of both pools and the
    rows behind the last token unchanged; separate tensors and a joint
    projection's slices."""
    import torch
    T, H, HK, D, rot, B, dtype, norm, inter, far = case
    c = make(case, T * 31 + rot + joint, joint)
    t = lambda a: None if a is None else torch.from_numpy(a).cuda()  # noqa: E731
    if joint:
        qkv = to_dev(c["qkv"], dtype)
        q = qkv[:, :H * D].view(T, H, D)
        k = qkv[:, H * D:(H + HK) * D].view(T, HK, D)
        v = qkv[:, (H + HK) * D:(H + 2 * HK) * D].view(T, HK, D)
    else:
        q, k, v = (to_dev(np.ascontiguousarray(c[n]), dtype) for n in "qkv")
    slots = c["slots"].copy()
    if T > 4:
        slots[2], slots[4] = -1, -7                      # not written, still turned
    kc, vc = to_dev(c["kc"], dtype), to_dev(c["vc"], dtype)
    out = torch.full((T + 2, H, D), 7.0, dtype=q.dtype, device="cuda")
    eps, rs = 1e-5, 1.25
    phases = pkv.rope_phases(c["f"]) if rot else None
    pkv.norm_rope_and_cache(out[:T], q, k, v, kc, vc, t(slots), t(c["pos"]), phases,
                            q_weight=t(c["qw"]), k_weight=t(c["kw"]), eps=eps, rope_scale=rs,
                            interleaved=inter)
    assert pkv.get_device_error() == 0
    assert (out[T:] == 7.0).all()
    check(out[:T], f64(np.ascontiguousarray(c["q"]), dtype), c["pos"], c["f"], c["qw"], eps, rs,
          inter, dtype, "q")
    kg, vg, vref = W.torch_to_words(kc), W.torch_to_words(vc), c["vc"].copy()
    live = np.flatnonzero(slots >= 0)
    blk, off = slots[live] // B, slots[live] % B
    rows = W.words_to_torch(np.ascontiguousarray(kg[blk, :, off]), dtype)
    check(rows, f64(np.ascontiguousarray(c["k"][live]), dtype), c["pos"][live], c["f"], c["kw"],
          eps, rs, inter, dtype, "k")
    kg[blk, :, off] = c["kc"][blk, :, off]               # every other slot as it was
    assert np.array_equal(kg, c["kc"])
    vref[blk, :, off] = c["v"][live]
    assert np.array_equal(vg, vref)


def test_in_place_negative_position_and_special_values(pkv):
    """q_out may be q; a negative position turns backwards; values keep their
    bits (infinities, NaN payloads); a NaN or an infinity stays in its row."""
    import torch
    rs = np.random.default_rng(8)
    T, H, HK, D, B = 5, 3, 2, 128, 16
    q, k = words((T, H, D), "f16", rs), words((T, HK, D), "f16", rs)
    v = rs.integers(0, 1 << 16, size=(T, HK, D)).astype(np.uint16)
    q[1, 0, 5], q[2, 2, 7] = 0x7E01, 0x7C00              # NaN, infinity
    kc, vc = np.zeros((1, HK, B, D), np.uint16), np.zeros((1, HK, B, D), np.uint16)
    pos = np.array([-1000, 5, 6, 2 ** 31 - 1, -2 ** 31], np.int32)
    f = 10000.0 ** (-np.arange(0, 64, 2) / 64)
    dq, dkc, dvc = to_dev(q, "f16"), to_dev(kc, "f16"), to_dev(vc, "f16")
    args = (to_dev(k, "f16"), to_dev(v, "f16"), dkc, dvc, torch.arange(T, device="cuda"),
            torch.from_numpy(pos).cuda(), pkv.rope_phases(f))
    out = torch.empty_like(dq)
    pkv.norm_rope_and_cache(out, dq, *args)
    pkv.norm_rope_and_cache(dq, dq, *args)
    assert torch.equal(out.view(torch.int16), dq.view(torch.int16))
    good = np.ones((T, H), bool)
    good[1, 0] = good[2, 2] = False
    x = f64(q, "f16")
    ref = norm_rope(np.where(good[..., None], x, 0.0), pos, f)
    lim = bound(np.where(good[..., None], x, 0.0), ref, pos, f, None, 0, 1.0, False, "f16")
    g = out.double().cpu().numpy()
    assert (np.abs(g - ref) <= lim)[good].all()
    assert np.isnan(g[1, 0, [5, 37]]).all() and np.isnan(g[1, 0]).sum() == 2
    assert np.array_equal(W.torch_to_words(dvc)[0, :, :T].transpose(1, 0, 2), v)


def test_bad_slots_are_skipped_and_flagged(pkv):
    import torch
    from paged_kv_cache_05_gb300.pagedkv import DEVERR_BAD_SLOT
    rs = np.random.default_rng(9)
    T, H, HK, D, B, nb = 3, 2, 1, 64, 16, 2
    x = [to_dev(words(s, "bf16", rs), "bf16") for s in ((T, H, D), (T, HK, D), (T, HK, D))]
    kc, vc = (to_dev(words((nb, HK, B, D), "bf16", rs), "bf16") for _ in range(2))
    k0, v0 = kc.clone(), vc.clone()
    pos = torch.arange(T, device="cuda", dtype=torch.int32)
    ph = pkv.rope_phases(pkv.rope_inv_freq(D)[0])
    want = torch.empty_like(x[0])
    pkv.norm_rope_and_cache(want, *x, kc.clone(), vc.clone(),
                            torch.arange(T, device="cuda"), pos, ph)
    out = torch.empty_like(x[0])
    bad = torch.tensor([nb * B, -1, 2 ** 62], device="cuda")
    pkv.norm_rope_and_cache(out, *x, kc, vc, bad, pos, ph)
    assert pkv.get_device_error() == DEVERR_BAD_SLOT and pkv.get_device_error() == 0
    assert torch.equal(out, want) and torch.equal(kc, k0) and torch.equal(vc, v0)


def test_captured_replayed_and_on_another_stream(pkv):
    """The call in a graph, replayed after its inputs changed, and on a stream of
    its own, gives what the plain call gives."""
    import torch
    rs = np.random.default_rng(10)
    case = (40, 8, 2, 128, 128, 16, "bf16", "qk", False, 5000)
    T, H, HK, D, rot, B, dtype = case[:7]
    c = make(case, 1, False)
    q, k, v = (to_dev(np.ascontiguousarray(c[n]), dtype) for n in "qkv")
    kc, vc = to_dev(c["kc"], dtype), to_dev(c["vc"], dtype)
    pos, slots = torch.from_numpy(c["pos"]).cuda(), torch.from_numpy(c["slots"]).cuda()
    qw, kw = (torch.from_numpy(c[n]).cuda() for n in ("qw", "kw"))
    ph, out = pkv.rope_phases(c["f"]), torch.empty_like(q)
    call = lambda s=None: pkv.norm_rope_and_cache(  # noqa: E731
        out, q, k, v, kc, vc, slots, pos, ph, q_weight=qw, k_weight=kw, stream=s)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    call(side)
    side.synchronize()
    first = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for shift in (0, 3):
        pos.add_(shift)
        out.zero_()
        graph.replay()
        got, pool = out.clone(), kc.clone()
        out.zero_()
        call()
        assert torch.equal(got, out) and torch.equal(pool, kc)
        assert torch.equal(got, first) == (shift == 0)


def test_long_context_scalings_reach_the_kernel(pkv):
    """by_parts frequencies and their scale factor, as a user passes them."""
    import torch
    rs = np.random.default_rng(11)
    T, H, D, B = 9, 2, 64, 8
    q, k = words((T, H, D), "f16", rs), words((T, H, D), "f16", rs)
    pos = rs.integers(0, 65536, size=T).astype(np.int32)
    f, scale = pkv.rope_inv_freq(D, 10000.0, "by_parts", 8.0, 8192)
    assert math.isclose(scale, 0.1 * math.log(8.0) + 1.0, rel_tol=1e-6)
    kc = torch.zeros((2, H, B, D), dtype=torch.float16, device="cuda")
    out = torch.empty((T, H, D), dtype=torch.float16, device="cuda")
    pkv.norm_rope_and_cache(out, to_dev(q, "f16"), to_dev(k, "f16"), to_dev(k, "f16"), kc,
                            kc.clone(), torch.arange(T, device="cuda"),
                            torch.from_numpy(pos).cuda(), pkv.rope_phases(f), rope_scale=scale)
    check(out, f64(q, "f16"), pos, f, None, 0, scale, False, "f16", "q")
