"""The latent attention kernels' waits keep the limit that is set and report running out; what
they had in flight ends first, and the next call is right."""
import time

import numpy as np
import pytest

from latent_helpers import (check_decode, check_prefill, decode_case, on_device, prefill_case,
                            run_decode, run_prefill)

pytestmark = pytest.mark.gpu

LIMITS = [0, 500, 1000, 2000, 4000, 8000, 16000]        # ns: from the first wait on to hardly any


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_05_gb300 import build
    build.build()
    import paged_kv_cache_05_gb300 as m
    return m


def under_limits(pkv, call, good):
    """The limits in turn, twice each: a call that runs out reports that and nothing else, one
    that does not is right; with the limit as it was every call is.  What is waited for at the
    end, whatever the limit, comes: waiting for something else would take the 1 s bound."""
    import torch
    from paged_kv_cache_05_gb300.pagedkv import DEVERR_TIMEOUT
    for ns in LIMITS:
        seen = 0
        for _ in range(2):
            before = pkv.set_decode_wait_limit(ns)
            try:
                torch.cuda.synchronize()
                t = time.perf_counter()
                got = call()
                bits = pkv.get_device_error(clear=True)
                t = time.perf_counter() - t
            finally:
                pkv.set_decode_wait_limit(before)
            assert bits in (0, DEVERR_TIMEOUT) and t < 0.9
            assert bits or torch.equal(got, good)
            seen |= bits
        assert ns or seen == DEVERR_TIMEOUT
        assert torch.equal(call(), good)
        assert pkv.get_device_error() == 0


@pytest.mark.parametrize("H,R,new,ctx,dtype", [
    (16, 512, [1] * 8, [8000 - 700 * i for i in range(8)], "bf16"),
    (128, 512, [1] * 3, [700, 1, 130], "f16"),
    (20, 256, [3, 1], [4000, 90], "f16"),
    (128, 256, [4] * 6, [1500, 300, 64, 2000, 5, 900], "bf16"),        # tiles of 256 rows
])
def test_absorbed(pkv, H, R, new, ctx, dtype):
    rs = np.random.RandomState(H + R)
    c = decode_case(rs, H, R, 16, new, ctx, dtype)
    good = check_decode(pkv, c, 0.07)
    d = on_device(c)
    under_limits(pkv, lambda: run_decode(pkv, c, 0.07, d), good)


@pytest.mark.parametrize("H,N,new,keys,dtype", [
    (4, 128, [300, 1, 130], [300, 200, 512], "bf16"),                  # whole items
    (4, 64, [600, 40, 257], [1300, 900, 257], "f16"),
    (16, 128, [700, 300], [1000, 1024], "bf16"),
])
def test_expanded(pkv, H, N, new, keys, dtype):
    rs = np.random.RandomState(H + N)
    c = prefill_case(rs, H, N, new, keys, dtype)
    scale = (N + 64) ** -0.5
    good = check_prefill(pkv, c, scale)
    under_limits(pkv, lambda: run_prefill(pkv, c, scale), good)
