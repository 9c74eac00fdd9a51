"""Short prompts in tables far wider than they need, as servers keep: the same
answers with a workspace, without one and in a narrow table."""
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


@pytest.mark.parametrize("H,HK,D,new,ctx,cap,biased", [
    (32, 8, 128, [61], [61], 0.0, False),
    (8, 2, 64, [125, 1, 0, 40], [125, 9, 0, 300], 30.0, False),
    (6, 1, 128, [3, 7], [900, 20], 0.0, True),
    (4, 4, 64, [200], [260], 1e6, False),
])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_wide_tables(pkv, H, HK, D, new, ctx, cap, biased, dtype):
    import torch
    B, S = 16, len(new)
    c = make_case(np.random.default_rng(H + D), H, HK, D, B, new, ctx, dtype, 0, 2.0)
    slopes = (2.0 ** (-8.0 * np.arange(1, H + 1) / H)).astype(np.float32) if biased else None
    ref, slack = reference(c, 0.1, cap, slopes)
    if 0 < cap <= 64:                     # the cap's form: 2^-20 of it, twice, over 2^-16
        slack = slack * (1 + cap / 8)
    if dtype == "f16":                    # weights of 11 bits
        slack = slack * (1 + 2.0 ** 5) + max(ctx) * 2.0 ** -25 * 6
    d = on_device(c)
    sl = None if slopes is None else torch.from_numpy(slopes).cuda()
    narrow = d["bt"]
    wide = torch.full((S, 2048), -1, dtype=torch.int32, device="cuda")
    wide[:, :narrow.shape[1]] = narrow
    none = torch.empty(0, dtype=torch.uint8, device="cuda")
    assert pkv.prefill_grouped_workspace_size(S, H, HK, D, B, 2048, max(new)) > 0
    outs = []
    for table, space in ((narrow, none), (wide, none), (wide, None)):
        out = torch.full_like(d["q"], 7.0)
        pkv.paged_attention_prefill_grouped(out, d["q"], d["kc"], d["vc"], table, d["cl"], d["qs"],
                                            0.1, max(new), softcap=cap, slopes=sl, workspace=space)
        assert pkv.get_device_error() == 0
        check(out, c, ref, slack)
        outs.append(out.view(torch.int16))
    # without a workspace the table's width is of no account (an uncapped fp16 call
    # with a K/V head per query head has the plain call's bits up to 8192 tokens only)
    assert torch.equal(outs[0], outs[1])
