"""Calls of the latent attention operators that take their rarer branches: outputs at addresses that
are multiples of 16 bytes only, parts of prompts far behind the first sequences, blocks past the
pool in either half of a step of 256-row tiles."""
import numpy as np
import pytest

import oracle.latent as L
from helpers import to_dev
from latent_helpers import (P, check, check_prefill, decode_case, f64, on_device, prefill_case,
                            run_decode)
from paged_kv_cache_05_gb300 import workloads as W

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_05_gb300 import build
    build.build()
    import paged_kv_cache_05_gb300 as m
    return m


def off_by_16_bytes(shape, dtype):
    """Contiguous, 16 bytes past a multiple of 32, with what lies around it."""
    import torch
    n = int(np.prod(shape))
    buf = torch.full((n + 16,), 7.0, dtype=W.torch_dtype(dtype), device="cuda")
    t = buf[8:8 + n].view(shape)
    assert t.data_ptr() % 32 == 16
    return t, buf


@pytest.mark.parametrize("H,R,new,ctx,dtype", [
    (16, 512, [1, 1], [100, 3000], "bf16"), (3, 256, [2, 5], [90, 1500], "f16"),
    (100, 256, [3, 3], [70, 2000], "bf16")])
def test_absorbed_to_16_bytes(pkv, H, R, new, ctx, dtype):
    import torch
    c = decode_case(np.random.RandomState(H), H, R, 16, new, ctx, dtype)
    d = on_device(c)
    want = run_decode(pkv, c, 0.07, d)
    assert want.data_ptr() % 32 == 0
    out, buf = off_by_16_bytes(want.shape, dtype)
    pkv.latent_attention_decode(out, d["q"], d["cache"], d["bt"], d["cl"], 0.07, query_start=d["qs"],
                                max_query_len=max(new))
    assert pkv.get_device_error() == 0
    assert torch.equal(out, want) and (buf[:8] == 7.0).all() and (buf[-8:] == 7.0).all()


@pytest.mark.parametrize("N", [64, 128])
@pytest.mark.parametrize("new,keys", [([50, 300], [60, 400]), ([700, 5], [900, 1300])])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_expanded_to_16_bytes(pkv, N, new, keys, dtype):
    import torch
    H = 3
    c = prefill_case(np.random.RandomState(N), H, N, new, keys, dtype)
    q, up, rows = (to_dev(c[n], dtype) for n in ("q", "up", "rows"))
    starts = [torch.from_numpy(c[n]).cuda() for n in ("qs", "ks")]
    want = torch.empty((sum(new), H, N), dtype=q.dtype, device="cuda")
    assert want.data_ptr() % 32 == 0
    out, buf = off_by_16_bytes(want.shape, dtype)
    for t in (want, out):
        pkv.latent_attention_prefill(t, q[:sum(new)], up[..., :N], rows[:, c["pad"]:], up[..., N:],
                                     *starts, 0.1, max(new), max(keys))
    assert pkv.get_device_error() == 0
    assert torch.equal(out, want) and (buf[:8] == 7.0).all() and (buf[-8:] == 7.0).all()


@pytest.mark.parametrize("N,dtype", [(64, "bf16"), (128, "f16")])
def test_cut_prompts_behind_many(pkv, N, dtype):
    """More sequences than a block has threads, the long ones, which are cut, among the last."""
    rs = np.random.RandomState(N)
    new = rs.randint(0, 9, 560).tolist()
    keys = [n + int(rs.randint(0, 9)) for n in new]
    for s, n, k in ((430, 3, 1500), (500, 540, 700), (559, 1, 2500)):
        new[s], keys[s] = n, k
    check_prefill(pkv, prefill_case(rs, 2, N, new, keys, dtype), (N + 64) ** -0.5)


@pytest.mark.parametrize("R,H", [(256, 100), (256, 20), (512, 16)])
@pytest.mark.parametrize("block", [0, 3, 5, 15])
def test_blocks_past_the_pool_are_left_out(pkv, R, H, block):
    """Blocks of 16 tokens, eight a step of 128, in its first half and its second; the rest of the
    tokens are attended as if the block's were not there."""
    c = decode_case(np.random.RandomState(block), H, R, 16, [3], [300], "bf16")
    d = on_device(c)
    d["bt"][0, block] = c["nb"] + 3
    got = run_decode(pkv, c, 0.07, d)
    assert pkv.get_device_error(clear=True) == 1
    rows = f64(c["cache"], "bf16")[c["bt"][0, :19]].reshape(-1, R + P)
    q = f64(c["q"], "bf16")
    t = np.arange(300)
    for i in range(3):
        see = rows[:300][(t <= 297 + i) & (t // 16 != block)]
        p = L._softmax(0.07 * q[i] @ see.T)
        ref, size = p @ see[:, :R], p @ np.abs(see[:, :R])
        big = float((np.abs(q[i]) @ np.abs(see).max(0)).max())
        dz = (R + P) / 16 * 2.0 ** -23 * 0.07 * big + 48 * 2.0 ** -20
        check(got[i], ref, "bf16", dz, size, 300, (block, i))
