"""Latent cache: norm, rotation and write of new tokens, and the gather of cached
rows, against the fp64 definitions."""
import numpy as np
import pytest

import oracle.latent as L
from helpers import to_dev, words
from latent_helpers import P, f64, half_step
from oracle.grouped import norm_rope
from paged_kv_cache_05_gb300 import workloads as W

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_05_gb300 import build
    build.build()
    import paged_kv_cache_05_gb300 as m
    return m


def near(got, ref, dtype, scale, what):
    """fp32 arithmetic of a few operations (2^-20 of the pair's or row's size), one rounding."""
    g = got.double().cpu().numpy()
    lim = half_step(dtype) * np.abs(ref) + 2.0 ** -20 * scale + (2.0 ** -25 if dtype == "f16" else 0)
    assert (np.abs(g - ref) <= lim).all(), what


@pytest.mark.parametrize("T,H,R,B,dtype,norm,interleaved,in_place", [
    (1, 1, 512, 16, "bf16", True, True, False),
    (1, 16, 512, 8, "f16", True, False, True),
    (7, 128, 256, 64, "bf16", False, True, True),
    (64, 3, 512, 32, "f16", True, True, False),
    (133, 20, 256, 16, "bf16", True, False, False),
    (2500, 5, 512, 64, "f16", False, False, True),
])
def test_write(pkv, T, H, R, B, dtype, norm, interleaved, in_place):
    import torch
    rs = np.random.RandomState(T + H)
    down, query = words((T, R + P), dtype, rs), words((T, H, 32 + P), dtype, rs)
    nb = -(-T // B) + 2
    cache0 = words((nb, B, R + P), dtype, rs)
    slots = rs.permutation(nb * B)[:T].astype(np.int64)
    if T > 3:
        slots[2] = -1
    pos = rs.randint(0, 200000, T).astype(np.int32)
    freq, rscale = pkv.rope_inv_freq(P, 500000.0, "by_parts", 8.0, 4096)
    phases = pkv.rope_phases(freq)
    weight = rs.uniform(0.5, 1.5, R).astype(np.float32) if norm else None
    d, qd, cache = to_dev(down, dtype), to_dev(query, dtype), to_dev(cache0, dtype)
    q_out = qd[..., 32:] if in_place else torch.full((T, H, R + P), 3.0, dtype=qd.dtype,
                                                     device="cuda")[..., R:]
    pkv.latent_norm_rope_and_cache(
        q_out, qd[..., 32:], d[:, :R], d[:, R:], cache, torch.from_numpy(slots).cuda(),
        torch.from_numpy(pos).cuda(), phases, None if weight is None else torch.from_numpy(weight).cuda(),
        1e-6, rscale, interleaved)
    assert pkv.get_device_error() == 0
    x = f64(query, dtype)[..., 32:]
    near(q_out, norm_rope(x, pos, freq, rope_scale=rscale, interleaved=interleaved), dtype,
         8 * rscale, "queries")
    rows = L.cache_rows(f64(down, dtype)[:, :R], f64(down, dtype)[:, R:], pos, freq, weight, 1e-6,
                        rscale, interleaved)
    want = f64(cache0, dtype).reshape(-1, R + P)
    live = slots >= 0
    want[slots[live]] = rows[live]
    got = cache.reshape(-1, R + P)
    near(got, want, dtype, 8 * rscale, "cache")
    untouched = np.ones(nb * B, bool)
    untouched[slots[live]] = False
    assert np.array_equal(W.torch_to_words(got.cpu())[untouched],
                          cache0.reshape(-1, R + P)[untouched])
    if weight is None:                             # the latent is a bit copy
        assert np.array_equal(W.torch_to_words(got.cpu())[slots[live]][:, :R], down[live][:, :R])
    if in_place:                                   # what lies beside the rotary parts stays
        assert np.array_equal(W.torch_to_words(qd.cpu())[..., :32], query[..., :32])


def test_write_bad_slot(pkv):
    import torch
    z = lambda *s: torch.zeros(s, dtype=torch.float16, device="cuda")  # noqa: E731
    cache = z(2, 8, 320)
    phases = pkv.rope_phases(pkv.rope_inv_freq(P)[0])
    q = torch.ones(2, 3, P, dtype=torch.float16, device="cuda")
    q_out = z(2, 3, P)
    pkv.latent_norm_rope_and_cache(q_out, q, torch.ones_like(z(2, 256)), torch.ones_like(z(2, P)),
                                   cache, torch.tensor([16, 5], device="cuda"),
                                   torch.zeros(2, dtype=torch.int32, device="cuda"), phases)
    assert pkv.get_device_error() == 2             # BAD_SLOT
    assert torch.equal(q_out, q)                   # position 0 turns nothing
    assert (cache.view(16, 320)[5] == 1).all() and cache.sum() == 320


@pytest.mark.parametrize("lens,R,B,dtype", [
    ([1], 512, 16, "bf16"), ([0, 5, 0, 0, 17, 0], 256, 8, "f16"), ([700], 512, 64, "f16"),
    ([33, 1, 0, 257, 64], 512, 32, "bf16"), ([3001, 1999], 256, 16, "bf16"), ([0, 0], 512, 16, "f16"),
])
def test_gather(pkv, lens, R, B, dtype):
    import torch
    rs = np.random.RandomState(len(lens) + R)
    need = [-(-n // B) for n in lens]
    nb = sum(need) + 2
    cache = words((nb, B, R + P), dtype, rs)
    tables = np.full((len(lens), max(need) + 1), nb + 7, np.int32)
    perm, at = rs.permutation(nb), 0
    for s, n in enumerate(need):
        tables[s, :n] = perm[at:at + n]
        at += n
    # two rows before the first sequence's and three after the last's
    start = (2 + np.concatenate([[0], np.cumsum(lens)])).astype(np.int32)
    rows = torch.full((int(start[-1]) + 3, R + P), 7.0, dtype=W.torch_dtype(dtype), device="cuda")
    pkv.gather_latent(rows, to_dev(cache, dtype), torch.from_numpy(tables).cuda(),
                      torch.from_numpy(start).cuda())
    assert pkv.get_device_error() == 0
    want = np.concatenate([cache[tables[s, :need[s]]].reshape(-1, R + P)[:n]
                           for s, n in enumerate(lens)] or [np.zeros((0, R + P), np.uint16)])
    got = W.torch_to_words(rows.cpu())
    assert np.array_equal(got[2:2 + sum(lens)], want)
    assert (rows[:2] == 7).all() and (rows[2 + sum(lens):] == 7).all()


def test_gather_reports_bad_blocks_and_lengths(pkv):
    import torch
    cache = torch.ones(3, 8, 320, dtype=torch.float16, device="cuda")
    rows = torch.zeros(20, 320, dtype=torch.float16, device="cuda")
    tables = torch.tensor([[0, 9], [-4, 2]], dtype=torch.int32, device="cuda")
    pkv.gather_latent(rows, cache, tables, torch.tensor([0, 10, 20], dtype=torch.int32, device="cuda"))
    assert pkv.get_device_error() == 1             # BAD_BLOCK
    assert rows.sum(1).eq(320).cpu().tolist() == [True] * 8 + [False] * 10 + [True] * 2
    rows.zero_()
    pkv.gather_latent(rows, cache, torch.tensor([[0, 1]], dtype=torch.int32, device="cuda"),
                      torch.tensor([0, 18], dtype=torch.int32, device="cuda"))
    assert pkv.get_device_error() == 4             # BAD_CONTEXT
    assert rows.sum(1).eq(320).cpu().tolist() == [True] * 16 + [False] * 4
