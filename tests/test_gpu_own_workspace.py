"""The workspace that a call takes for itself, on a stream that is not the current
one: memory that the current stream has given back while its work on it is still
pending must not be handed to the call."""
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


def pending(size, call):
    """Runs `call(stream)` on another stream while the current one has yet to read a
    buffer of `size` bytes that was given back; what it then read."""
    import torch
    side = torch.cuda.Stream()
    call(side)                                     # loaded and warm
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    kept = torch.zeros(size, dtype=torch.uint8, device="cuda")
    buf = torch.full((size,), 0x5A, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)                 # about 0.1 s
    kept.copy_(buf)
    del buf
    call(side)
    side.synchronize()
    torch.cuda.synchronize()
    return kept


def batch(H, HK, D, new, ctx, dtype="f16"):
    c = make_case(np.random.default_rng(23), H, HK, D, 16, new, ctx, dtype, wild=False)
    ref, slack = reference(c, 0.09, 0.0, None)
    if dtype == "f16":                             # weights of 11 bits
        slack = slack * (1 + 2.0 ** 5) + max(ctx) * 2.0 ** -25 * 6
    return c, on_device(c), ref, slack


def test_grouped_prompts(pkv):
    import torch
    c, d, ref, slack = batch(8, 2, 128, [6, 9], [2600, 1900])
    size = pkv.prefill_grouped_workspace_size(2, 8, 2, 128, 16, c["bt"].shape[1], 9)
    assert size > 0
    out = torch.empty_like(d["q"])
    kept = pending(size, lambda s: pkv.paged_attention_prefill_grouped(
        out, d["q"], d["kc"], d["vc"], d["bt"], d["cl"], d["qs"], 0.09, 9, stream=s))
    assert (kept == 0x5A).all()
    check(out, c, ref, slack)
    assert pkv.get_device_error() == 0


def test_grouped_prompts_on_the_default_stream(pkv):
    """The call's stream is the default one, the current one another."""
    import torch
    c, d, ref, slack = batch(8, 2, 128, [6, 9], [2600, 1900])
    out = torch.empty_like(d["q"])
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        pkv.paged_attention_prefill_grouped(out, d["q"], d["kc"], d["vc"], d["bt"], d["cl"],
                                            d["qs"], 0.09, 9, stream=torch.cuda.default_stream())
    torch.cuda.synchronize()
    check(out, c, ref, slack)


def test_grouped_decode(pkv):
    import torch
    c, d, ref, slack = batch(8, 2, 128, [1] * 3, [2600, 1900, 5])
    size = pkv.decode_grouped_workspace_size(3, 8, 2, 128, 16, c["bt"].shape[1])
    out = torch.empty_like(d["q"])
    kept = pending(size, lambda s: pkv.paged_attention_decode_grouped(
        out, d["q"], d["kc"], d["vc"], d["bt"], d["cl"], 0.09, stream=s))
    assert (kept == 0x5A).all()
    check(out, c, ref, slack)
    assert pkv.get_device_error() == 0


@pytest.mark.parametrize("which", ["decode", "append", "shared", "contiguous"])
def test_decode_calls(pkv, which):
    """The calls for one K/V head per query head."""
    import torch
    H, D, B, n, S = 4, 128, 16, 4000, 2
    c, d, ref, slack = batch(H, H, D, [1] * S, [n] * S)
    mb = c["bt"].shape[1]
    out = torch.empty_like(d["q"])
    if which == "shared":
        size = pkv.decode_shared_workspace_size(S, H, D, B, mb)
        call = lambda s: pkv.paged_attention_decode_shared(  # noqa: E731
            out, d["q"], d["kc"], d["vc"], d["bt"], d["cl"], 0.09, stream=s)
    elif which == "contiguous":
        k, v = (p[d["bt"][:, :n // B].long()].transpose(1, 2).reshape(S, H, n, D).contiguous()
                for p in (d["kc"], d["vc"]))
        size = pkv.contiguous_workspace_size(S, H, D, n)
        call = lambda s: pkv.contiguous_attention_decode(  # noqa: E731
            out, d["q"], k, v, d["cl"], 0.09, stream=s)
    else:
        size = pkv.decode_workspace_size(S, H, D, B, mb)
        at = (d["bt"][:, (n - 1) // B].long(), slice(None), (n - 1) % B)
        new = [d[p][at].contiguous() for p in ("kc", "vc")] if which == "append" else []
        f = pkv.paged_attention_decode_append if new else pkv.paged_attention_decode
        call = lambda s: f(out, d["q"], *new, d["kc"], d["vc"], d["bt"], d["cl"], 0.09,  # noqa: E731
                           stream=s)
    kept = pending(max(size, 256), call)
    assert (kept == 0x5A).all()
    check(out, c, ref, slack)
    assert pkv.get_device_error() == 0
