"""Absorbed latent attention of latent 256 with more than 192 rows a sequence on average, which
takes tiles of 256 rows, and its neighbours that take tiles of 128."""
import numpy as np
import pytest

from latent_helpers import check_decode, decode_case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_05_gb300 import build
    build.build()
    import paged_kv_cache_05_gb300 as m
    return m


@pytest.mark.parametrize("H,B,new,ctx,dtype,tree", [
    (20, 32, [13, 13, 13], [200, 1300, 13], "f16", True),        # 260 rows: a tile and 4 rows
    (64, 16, [4], [4], "bf16", False),                           # a whole tile, one step
    (64, 16, [3, 3], [129, 640], "f16", False),                  # exactly 192 rows: tiles of 128
    (65, 8, [3, 3], [127, 128], "f16", False),                   # three rows more
    (128, 64, [2, 1, 5], [33, 1, 700], "bf16", False),           # 128 live rows: one CTA of a pair
    (2, 16, [0, 400, 0], [0, 500, 90], "bf16", False),           # four tiles, empty places
    (7, 16, [64, 64], [64, 2500], "f16", True),
    (100, 16, [9], [3000], "bf16", False),                       # cut among many pairs
])
def test_shapes(pkv, H, B, new, ctx, dtype, tree):
    rs = np.random.RandomState(H + sum(ctx))
    check_decode(pkv, decode_case(rs, H, 256, B, new, ctx, dtype, tree), 320 ** -0.5)


@pytest.mark.parametrize("dtype,qtimes", [("f16", 30.0), ("bf16", 30.0), ("f16", 0.01)])
def test_sharp_and_flat_scores(pkv, dtype, qtimes):
    rs = np.random.RandomState(31)
    check_decode(pkv, decode_case(rs, 64, 256, 16, [4, 4], [900, 333], dtype, qtimes=qtimes), 0.07)


def test_rows_that_see_nothing_and_bad_blocks(pkv):
    """Trees whose rows have no bits and no tokens before them are 0; a block past the pool is
    left out and reported, other sequences keep their bits."""
    import torch
    from latent_helpers import on_device, run_decode
    rs = np.random.RandomState(32)
    c = decode_case(rs, 100, 256, 16, [5, 3], [5, 700], "bf16", tree=True)
    c["tree"][0] = 0
    got = check_decode(pkv, c, 0.07)
    assert (got[0] == 0).all() and (got[1:] != 0).any()
    d = on_device(c)
    d["bt"][1, 3] = c["nb"] + 5
    bad = run_decode(pkv, c, 0.07, d)
    bits = pkv.get_device_error(clear=True)
    assert bits == 1
    assert torch.equal(bad[:5], got[:5]) and torch.isfinite(bad).all()


def test_same_bits_and_workspace_size(pkv):
    import torch
    from latent_helpers import on_device, run_decode
    rs = np.random.RandomState(33)
    c = decode_case(rs, 128, 256, 16, [4, 4, 1], [1700, 300, 40], "f16")
    d = on_device(c)
    ws = pkv.alloc_latent_workspace(3, 128, 256, 4)
    first = run_decode(pkv, c, 0.07, d)
    for _ in range(3):
        assert torch.equal(first, run_decode(pkv, c, 0.07, d, workspace=ws))
    assert pkv.get_device_error() == 0
