"""Expanded latent attention of a call without any keys: rows of a sequence are reported, rows of
none (a padded batch) are not, and both are left as they are."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_05_gb300 import build
    build.build()
    import paged_kv_cache_05_gb300 as m
    return m


@pytest.mark.parametrize("N", [64, 128])
@pytest.mark.parametrize("starts,bad", [([0, 0, 0], False), ([0, 3, 3], True), ([2, 2, 5], True)])
@pytest.mark.parametrize("max_keys", [0, 7, 900])
def test_no_keys(pkv, N, starts, bad, max_keys):
    import torch
    from paged_kv_cache_05_gb300.pagedkv import DEVERR_BAD_CONTEXT
    H = 3
    t = dict(dtype=torch.float16, device="cuda")
    q = torch.ones((5, H, N + 64), **t)
    up = torch.empty((0, H, 2 * N), **t)
    out = torch.full((5, H, N), 7.0, **t)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")      # noqa: E731
    pkv.latent_attention_prefill(out, q, up[..., :N], torch.empty((0, 64), **t), up[..., N:],
                                 i32(starts), i32([0, 0, 0]), 0.1, 4, max_keys)
    assert pkv.get_device_error(clear=True) == (DEVERR_BAD_CONTEXT if bad else 0)
    assert (out == 7.0).all()
