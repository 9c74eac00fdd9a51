"""Runs of the latent attention kernels that end at every place of their rings, launched one
behind the other: each launch begins where CTAs of the one before have just gone."""
import numpy as np
import pytest

import oracle.latent as L
from latent_helpers import check, decode_case, decode_reference, f64, prefill_case, weighted_size
from helpers import to_dev
from paged_kv_cache_05_gb300 import workloads as W

pytestmark = pytest.mark.gpu

TIMES = 19                                   # by four: a run of its own for each of 76 pairs


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_05_gb300 import build
    build.build()
    import paged_kv_cache_05_gb300 as m
    return m


@pytest.mark.parametrize("H,R,dtype", [(4, 512, "bf16"), (200, 256, "f16"), (5, 256, "f16")])
@pytest.mark.parametrize("steps", [1, 2, 3, 4, 5, 8, 9])
def test_absorbed(pkv, H, R, dtype, steps):
    import torch
    rs = np.random.RandomState(H + steps)
    c = decode_case(rs, H, R, 16, [1] * 4, [128 * steps - n for n in (0, 3, 31, 97)], dtype)
    ref, dz = decode_reference(c, 0.07)
    size = weighted_size(c, 0.07)
    q, cache = (to_dev(c[n], dtype) for n in ("q", "cache"))
    q = q.repeat(TIMES, 1, 1)
    bt, cl = (torch.from_numpy(c[n]).cuda() for n in ("bt", "ctx"))
    bt, cl = bt.repeat(TIMES, 1), cl.repeat(TIMES)
    ws = pkv.alloc_latent_workspace(4 * TIMES, H, R)
    outs = [torch.full((4 * TIMES, H, R), 7.0, dtype=q.dtype, device="cuda") for _ in range(12)]
    for out in outs:
        pkv.latent_attention_decode(out, q, cache, bt, cl, 0.07, workspace=ws)
    assert pkv.get_device_error() == 0
    for out in outs[1:]:
        assert torch.equal(out, outs[0])
    for k in range(TIMES):
        check(outs[0][4 * k:4 * k + 4], ref, dtype, dz, size, int(max(c["ctx"])), k)


@pytest.mark.parametrize("N,dtype", [(128, "bf16"), (64, "f16")])
@pytest.mark.parametrize("new,keys", [(1, 1), (1, 70), (64, 128), (40, 180), (190, 250), (256, 300),
                                      (257, 384), (400, 440), (512, 512), (3, 1000), (600, 700)])
def test_expanded(pkv, N, dtype, new, keys):
    import torch
    rs = np.random.RandomState(N + keys)
    c = prefill_case(rs, 2, N, [new] * 2, [keys] * 2, dtype)
    full = {n: to_dev(c[n], dtype) for n in ("q", "up", "rows")}
    q = full["q"][:c["Tq"]].repeat(TIMES, 1, 1)
    up = full["up"][:2 * keys].repeat(TIMES, 1, 1)
    r = full["rows"][:2 * keys].repeat(TIMES, 1)
    starts = lambda n: torch.arange(2 * TIMES + 1, dtype=torch.int32, device="cuda") * n  # noqa: E731
    scale = (N + 64) ** -0.5
    ws = None
    if pkv.latent_prefill_workspace_size(N, new, keys):
        ws = torch.empty(pkv.latent_prefill_workspace_size(N, new, keys), dtype=torch.uint8, device="cuda")
    outs = [torch.full((q.shape[0], 2, N), 7.0, dtype=W.torch_dtype(dtype), device="cuda")
            for _ in range(12)]
    for out in outs:
        pkv.latent_attention_prefill(out, q, up[..., :N], r[:, c["pad"]:], up[..., N:], starts(new),
                                     starts(keys), scale, new, keys, workspace=ws)
    assert pkv.get_device_error() == 0
    for out in outs[1:]:
        assert torch.equal(out, outs[0])
    qd, ud, rd = (f64(c[n], dtype) for n in ("q", "up", "rows"))
    k, v, rd = ud[:2 * keys, :, :N], ud[:2 * keys, :, N:], rd[:2 * keys, c["pad"]:]
    qd = qd[:c["Tq"]]
    ref = L.prefill(qd, k, rd, v, c["qs"], c["ks"], scale)
    size = L.prefill(qd, k, rd, np.abs(v), c["qs"], c["ks"], scale)
    most = np.abs(k).max(0).sum(-1) + np.abs(rd).max(0).sum()
    dz = (N + 64) / 16 * 2.0 ** -23 * scale * float((np.abs(qd).max() * most).max()) + 48 * 2.0 ** -20
    for n in range(TIMES):
        check(outs[0][n * c["Tq"]:(n + 1) * c["Tq"]], ref, dtype, dz, size, keys, n)
