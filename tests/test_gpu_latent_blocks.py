"""Forks and swaps of sequences whose cache is latent: the block manager's pairs applied by
copy_blocks and swap_blocks to pools taken as [blocks, (R + 64) / 64, B, 64]."""
import numpy as np
import pytest

import oracle.latent as L
from helpers import to_dev, words
from latent_helpers import P, check, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_05_gb300 import build
    build.build()
    import paged_kv_cache_05_gb300 as m
    return m


def halves(pool):
    nb, B, W = pool.shape
    return pool.view(nb, W // 64, B, 64)


@pytest.mark.parametrize("R,B,dtype,alone", [(512, 16, "bf16", False), (256, 32, "f16", False),
                                             (512, 8, "f16", True)])
def test_forks_and_swaps(pkv, R, B, dtype, alone):
    """Two children of a prompt write a token each into the block they shared; then one is swapped
    out and back.  Every layer attends what its own sequence wrote."""
    import torch
    rs = np.random.RandomState(R + B)
    n, H, nb, layers = 5 * B + 3, 4, 40, 1 if alone else 2
    bm = pkv.BlockManager(nb, B, 3)
    pools = [torch.full((nb, B, R + P), float("nan"), dtype=to_dev(words((1,), dtype, rs), dtype).dtype,
                        device="cuda") for _ in range(layers)]
    rows = [words((n + 2, R + P), dtype, rs) for _ in range(layers)]
    slots = torch.from_numpy(bm.add_sequence(0, n)).cuda()
    for pool, r in zip(pools, rows):
        pool.view(-1, R + P)[slots] = to_dev(r[:n], dtype)
    bm.fork(0, 1)
    new, pairs = bm.append_slots([0, 1])
    assert len(pairs) == 1                       # the shared last block, copied for one of them
    two = (pools[0], pools[-1])
    pkv.copy_blocks(*map(halves, two), torch.from_numpy(pairs.copy()).cuda())
    for pool, r in zip(pools, rows):
        pool.view(-1, R + P)[torch.from_numpy(new).cuda()] = to_dev(r[n:], dtype)

    q = words((2, H, R + P), dtype, rs)

    def attend(ids):
        tables, ctx = bm.export(ids, 7)
        outs = []
        for pool in pools:
            out = torch.empty((len(ids), H, R), dtype=pool.dtype, device="cuda")
            outs.append(pkv.latent_attention_decode(out, to_dev(q[ids], dtype), pool,
                                                    torch.from_numpy(tables).cuda(),
                                                    torch.from_numpy(ctx).cuda(), 0.07))
        assert pkv.get_device_error() == 0
        return outs

    both = attend([0, 1])
    for out, r in zip(both, rows):
        for s in (0, 1):
            k = f64(np.concatenate([r[:n], r[n + s:n + s + 1]]), dtype)
            qd = f64(q[s:s + 1], dtype)
            keys = np.repeat(k[:, None], H, 1)
            # (the definition of the expanded form takes the latent part as the head's keys)
            ref = L.prefill(qd, keys[..., :R], k[:, R:], keys[..., :R], [0, 1], [0, n + 1], 0.07)
            size = L.prefill(qd, keys[..., :R], k[:, R:], np.abs(keys[..., :R]), [0, 1], [0, n + 1], 0.07)
            big = float((np.abs(qd) @ np.abs(k).max(0)).max())
            dz = (R + P) / 16 * 2.0 ** -23 * 0.07 * big + 48 * 2.0 ** -20
            check(out[s:s + 1], ref, dtype, dz, size, n + 1, s)

    bm.add_cpu_pool(nb, 5)
    host = [torch.zeros(pool.shape, dtype=pool.dtype).pin_memory() for pool in pools]
    hosts = (host[0], host[-1])
    out_pairs = bm.swap_out([0, 1])
    pkv.swap_blocks(*map(halves, hosts), *map(halves, two), torch.from_numpy(out_pairs.copy()).cuda())
    torch.cuda.synchronize()
    for pool in pools:
        pool.fill_(float("nan"))
    in_pairs = bm.swap_in([0, 1])
    pkv.swap_blocks(*map(halves, two), *map(halves, hosts), torch.from_numpy(in_pairs.copy()).cuda())
    for a, b in zip(attend([0, 1]), both):
        assert torch.equal(a, b)
