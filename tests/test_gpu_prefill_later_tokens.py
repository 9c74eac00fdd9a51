"""Tokens that no row of an item sees do not matter to it, not even those that
share a key tile or a block with tokens it sees."""
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


# H, HK, D, B, new, past, window, the token, tokens of an item (256 rows' worth)
CASES = [
    (4, 1, 64, 16, 300, 0, 0, 200, 64),
    (8, 1, 128, 8, 130, 70, 0, 147, 32),      # (position 147: new token 77)
    (16, 1, 64, 64, 100, 0, 60, 50, 16),
    (4, 4, 128, 32, 700, 0, 0, 530, 256),
]


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("dtype,cut", [("bf16", False), ("bf16", True), ("f16", False)])
def test_a_later_token_spoils_no_earlier_item(pkv, case, bad, dtype, cut):
    import torch
    H, HK, D, B, new, past, window, token, item = case
    S = 1 if cut else 3
    c = make_case(np.random.default_rng(H + D), H, HK, D, B, [new] * S, [new + past] * S, dtype,
                  window, wild=False)
    ref, slack = reference(c, 0.125, 0.0, None)
    if dtype == "f16":
        slack = slack * (1 + 2.0 ** 5) + (new + past) * 2.0 ** -25 * 6
    d = on_device(c)
    for s in range(S):
        at = (int(c["bt"][s, token // B]), slice(None), token % B)
        d["vc"][at] = bad
        d["kc"][at] = bad
    out = torch.empty_like(d["q"])
    space = None if cut else torch.empty(0, dtype=torch.uint8, device="cuda")
    pkv.paged_attention_prefill_grouped(out, d["q"], d["kc"], d["vc"], d["bt"], d["cl"], d["qs"],
                                        0.125, new, window=window, workspace=space)
    assert pkv.get_device_error() == 0
    before = (token - past) // item * item            # the rows of earlier items
    rows = np.concatenate([np.arange(before) + new * s for s in range(S)])
    check(out[torch.from_numpy(rows).cuda()], c, ref[rows], slack[rows])
