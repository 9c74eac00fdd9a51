"""The grouped decode's waits keep the limit that is set and report running out."""
import numpy as np
import pytest

from grouped_helpers import check, make_case, on_device, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_05_gb300 import build
    build.build()
    import paged_kv_cache_05_gb300 as m
    return m


def test_a_wait_that_runs_out_is_always_reported(pkv):
    """Without any time to wait: every ring has more steps than stages and its first
    copies take about a microsecond, so the copying warps find no free stage."""
    import torch
    from paged_kv_cache_05_gb300.pagedkv import DEVERR_TIMEOUT
    n, S, HK, B, D = 8192, 8, 8, 16, 128
    nb = S * n // B
    kc = torch.zeros((nb, HK, B, D), dtype=torch.bfloat16, device="cuda")
    q = torch.zeros((S, HK, D), dtype=torch.bfloat16, device="cuda")
    bt = torch.arange(nb, dtype=torch.int32, device="cuda").view(S, -1)
    cl = torch.full((S,), n, dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    before = pkv.set_decode_wait_limit(0)
    try:
        seen = 0
        for _ in range(4):
            pkv.paged_attention_decode_grouped(out, q, kc, kc, bt, cl, 0.1)
            seen |= pkv.get_device_error()
    finally:
        pkv.set_decode_wait_limit(before)
    assert seen == DEVERR_TIMEOUT
    c = make_case(np.random.default_rng(7), 8, 2, 128, 16, [1] * 8, [3000] * 8, "bf16", wild=False)
    ref, slack = reference(c, 0.1, 0.0, None)
    d = on_device(c)
    out = torch.empty_like(d["q"])
    pkv.paged_attention_decode_grouped(out, d["q"], d["kc"], d["vc"], d["bt"], d["cl"], 0.1)
    assert pkv.get_device_error() == 0
    check(out, c, ref, slack)
