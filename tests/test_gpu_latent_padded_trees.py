"""Trees padded to a fixed number of rows: places of drafted tokens that no row attends are never
written, and what they hold (NaN here) reaches no row."""
import numpy as np
import pytest

from latent_helpers import check_decode, decode_case, nan_word, run_decode

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_05_gb300 import build
    build.build()
    import paged_kv_cache_05_gb300 as m
    return m


def without(c, gone):
    """The case with the drafted tokens `gone` of every sequence attended by no row, their own
    rows attending nothing, and NaN in their places; and the same with 0 in them."""
    c["tree"] = list(c["tree"])
    zero = dict(c, cache=c["cache"].copy())
    for s, m in enumerate(c["new"]):
        for i in range(m):
            bits = c["tree"][c["qs"][s] + i]
            for g in gone:
                bits &= ~(1 << g)
            c["tree"][c["qs"][s] + i] = 0 if i in gone else bits
        for g in gone:
            if g < m:
                t = int(c["ctx"][s]) - m + g
                at = c["bt"][s, t // c["B"]], t % c["B"]
                c["cache"][at] = nan_word(c["dtype"])
                zero["cache"][at] = 0
    zero["tree"] = c["tree"]
    return c, zero


@pytest.mark.parametrize("H,R,B,new,ctx,dtype", [
    (16, 512, 16, [8, 8, 3], [300, 136, 131], "bf16"),
    (20, 256, 32, [13, 64, 9], [77, 400, 9], "f16"),
    (128, 256, 8, [8, 30], [700, 129], "bf16"),                # tiles of 256 rows
    (5, 512, 64, [64], [64], "f16"),
    (3, 256, 8, [64, 40], [2000, 168], "bf16"),
])
@pytest.mark.parametrize("gone", [[7], [0], [2, 3], list(range(5, 64)), list(range(0, 64, 3)),
                                  list(range(8, 16)), list(range(64))])
def test_unattended_places(pkv, H, R, B, new, ctx, dtype, gone):
    import torch
    rs = np.random.RandomState(H + len(gone))
    c, zero = without(decode_case(rs, H, R, B, new, ctx, dtype, tree=True), gone)
    got = run_decode(pkv, c, 0.07)
    assert pkv.get_device_error() == 0
    assert torch.equal(got, check_decode(pkv, zero, 0.07))


def test_waits_that_run_out(pkv):
    from latent_helpers import on_device
    from test_gpu_latent_waits import under_limits
    rs = np.random.RandomState(9)
    c, zero = without(decode_case(rs, 20, 256, 16, [40, 64, 30], [1000, 200, 700], "bf16", tree=True),
                      list(range(3, 64, 5)))
    good = check_decode(pkv, zero, 0.07)
    d = on_device(c)
    under_limits(pkv, lambda: run_decode(pkv, c, 0.07, d), good)
