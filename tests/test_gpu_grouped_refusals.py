"""What the grouped entry points refuse from Python: shapes, types, devices and
strides, before any launch; and what they take that may look odd."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_05_gb300 import build
    build.build()
    import paged_kv_cache_05_gb300 as m
    return m


def args(torch):
    dt, z = torch.float16, lambda *s, d=torch.float16: torch.zeros(s, dtype=d, device="cuda")
    write = dict(q_out=z(3, 4, 64), q=z(3, 4, 64), k=z(3, 2, 64), v=z(3, 2, 64),
                 k_cache=z(5, 2, 16, 64), v_cache=z(5, 2, 16, 64),
                 slot_mapping=torch.arange(3, device="cuda"), positions=z(3, d=torch.int32),
                 phases=z(32, d=torch.int64), q_weight=z(64, d=torch.float32),
                 k_weight=z(64, d=torch.float32))
    att = dict(out=z(3, 4, 64), q=z(3, 4, 64), k_cache=z(5, 2, 16, 64), v_cache=z(5, 2, 16, 64),
               block_tables=z(3, 2, d=torch.int32), context_lens=z(3, d=torch.int32) + 5,
               scale=0.1, slopes=z(4, d=torch.float32))
    pre = dict(att, context_lens=z(2, d=torch.int32) + 5, block_tables=z(2, 2, d=torch.int32),
               query_start=torch.tensor([0, 1, 3], dtype=torch.int32, device="cuda"),
               max_query_len=2)
    assert dt == write["q"].dtype
    return write, att, pre


def test_refusals(pkv):
    import torch
    write, att, pre = args(torch)
    pkv.norm_rope_and_cache(**write)
    pkv.paged_attention_decode_grouped(**att)
    pkv.paged_attention_prefill_grouped(**pre)
    assert pkv.get_device_error() == 0
    cases = [
        (pkv.norm_rope_and_cache, write, [
            ("q", lambda t: t.cpu(), ValueError), ("k", lambda t: t.bfloat16(), TypeError),
            ("q", lambda t: t.float(), TypeError), ("v", lambda t: t[:2], ValueError),
            ("k_cache", lambda t: t[:, :1], ValueError),
            ("v_cache", lambda t: t.transpose(0, 1), ValueError),
            ("q_out", lambda t: t[:, :2], ValueError),
            ("q_out", lambda t: t.permute(1, 0, 2).contiguous().permute(1, 0, 2), ValueError),
            ("q", lambda t: torch.zeros(3, 64, 4, dtype=t.dtype, device="cuda").mT, ValueError),
            ("k", lambda t: torch.zeros(3, 4, 64, dtype=t.dtype, device="cuda")[:, ::2], ValueError),
            ("slot_mapping", lambda t: t.int(), TypeError), ("slot_mapping", lambda t: t[:2], ValueError),
            ("positions", lambda t: t.long(), TypeError), ("positions", lambda t: t.cpu(), ValueError),
            ("phases", lambda t: t.double(), TypeError), ("phases", lambda t: t[:30], pkv.PagedKVError),
            ("phases", lambda t: t.view(2, 16), ValueError),
            ("q_weight", lambda t: t.half(), TypeError), ("k_weight", lambda t: t[:32], ValueError),
            ("q_out", lambda t: write["k"].new_zeros(3, 4, 64).cpu(), ValueError),
            ("q", lambda t: "q", TypeError),
        ]),
        (pkv.paged_attention_decode_grouped, att, [
            ("out", lambda t: t[:2], ValueError), ("out", lambda t: t.bfloat16(), TypeError),
            ("q", lambda t: t[:, :3].contiguous(), pkv.PagedKVError),
            ("block_tables", lambda t: t.long(), TypeError),
            ("block_tables", lambda t: t[0], ValueError),
            ("context_lens", lambda t: t[:1], ValueError),
            ("slopes", lambda t: t[:2], ValueError), ("slopes", lambda t: t.double(), TypeError),
            ("scale", lambda t: float("nan"), pkv.PagedKVError), ("scale", lambda t: "x", TypeError),
        ]),
        (pkv.paged_attention_prefill_grouped, pre, [
            ("query_start", lambda t: t[:2], ValueError), ("query_start", lambda t: t.cpu(), ValueError),
            ("max_query_len", lambda t: -1, pkv.PagedKVError),
            ("max_query_len", lambda t: 1 << 40, ValueError),
            ("context_lens", lambda t: t.view(2, 1), ValueError),
            ("k_cache", lambda t: t.bfloat16(), TypeError),
        ]),
    ]
    for fn, base, bad in cases:
        for name, change, error in bad:
            with pytest.raises(error):
                fn(**dict(base, **{name: change(base[name])}))
    for kw, error in ((dict(softcap=-1.0), pkv.PagedKVError), (dict(softcap=1e-45), pkv.PagedKVError),
                      (dict(window=-1), pkv.PagedKVError), (dict(window=1 << 31), ValueError)):
        with pytest.raises(error):
            pkv.paged_attention_decode_grouped(**dict(att, **kw))
        with pytest.raises(error):
            pkv.paged_attention_prefill_grouped(**dict(pre, **kw))
    small = torch.empty(64, dtype=torch.uint8, device="cuda")
    with pytest.raises(pkv.PagedKVError):
        pkv.paged_attention_decode_grouped(**att, workspace=small)
    # q_out shares memory with k
    both = torch.zeros(3, 6, 64, dtype=torch.float16, device="cuda")
    with pytest.raises(pkv.PagedKVError):
        pkv.norm_rope_and_cache(**dict(write, q_out=both.view(-1)[:768].view(3, 4, 64),
                                       k=both.view(-1)[640:1024].view(3, 2, 64)))
    torch.cuda.synchronize()
    assert pkv.get_device_error() == 0


def test_empty_batches_launch_nothing(pkv):
    import torch
    write, att, pre = args(torch)
    e = lambda t: t[:0]  # noqa: E731
    pkv.norm_rope_and_cache(**dict(write, **{n: e(write[n]) for n in (
        "q_out", "q", "k", "v", "slot_mapping", "positions")}))
    pkv.paged_attention_decode_grouped(**dict(att, **{n: e(att[n]) for n in (
        "out", "q", "block_tables", "context_lens")}))
    pkv.paged_attention_prefill_grouped(**dict(pre, out=e(pre["out"]), q=e(pre["q"])))
    assert pkv.get_device_error() == 0
