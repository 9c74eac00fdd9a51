"""What the latent entry points refuse from Python: shapes, types, devices, strides and
overlaps, before any launch; and empty batches."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_05_gb300 import build
    build.build()
    import paged_kv_cache_05_gb300 as m
    return m


def args(torch):
    z = lambda *s, d=torch.float16: torch.zeros(s, dtype=d, device="cuda")  # noqa: E731
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    write = dict(q_out=z(3, 4, 64), q=z(3, 4, 64), latent=z(3, 256), k_rope=z(3, 64),
                 cache=z(5, 16, 320), slot_mapping=torch.arange(3, device="cuda"),
                 positions=z(3, d=torch.int32), phases=z(32, d=torch.int64),
                 weight=z(256, d=torch.float32))
    gather = dict(rows=z(9, 320), cache=z(5, 16, 320), block_tables=z(2, 3, d=torch.int32),
                  key_start=i32(0, 4, 9))
    prompt = dict(out=z(3, 4, 128), q=z(3, 4, 192), k=z(7, 4, 128), k_rope=z(7, 64),
                  v=z(7, 4, 128), query_start=i32(0, 1, 3), key_start=i32(0, 4, 7), scale=0.1,
                  max_query_len=2, max_key_len=4)
    decode = dict(out=z(3, 4, 256), q=z(3, 4, 320), cache=z(5, 16, 320),
                  block_tables=z(2, 3, d=torch.int32), context_lens=i32(5, 9), scale=0.1,
                  query_start=i32(0, 1, 3), max_query_len=2, ancestors=z(3, d=torch.int64))
    return write, gather, prompt, decode


def test_refusals(pkv):
    import torch
    write, gather, prompt, decode = args(torch)
    E = pkv.PagedKVError
    pkv.latent_norm_rope_and_cache(**write)
    pkv.gather_latent(**gather)
    pkv.latent_attention_prefill(**prompt)
    pkv.latent_attention_decode(**decode)
    assert pkv.get_device_error() == 0
    wide = lambda t: torch.zeros(*t.shape[:-1], 2 * t.shape[-1], dtype=t.dtype, device="cuda")  # noqa: E731
    cases = [
        (pkv.latent_norm_rope_and_cache, write, [
            ("q", lambda t: t.cpu(), ValueError), ("q", lambda t: t.float(), TypeError),
            ("q", lambda t: t[:, :, :32], ValueError), ("q", lambda t: wide(t)[..., ::2], ValueError),
            ("latent", lambda t: t.bfloat16(), TypeError), ("latent", lambda t: t[:2], ValueError),
            ("latent", lambda t: t[:, :128], ValueError), ("latent", lambda t: t[0], ValueError),
            ("k_rope", lambda t: t[:, :32], ValueError),
            ("k_rope", lambda t: torch.zeros(3, 68, dtype=t.dtype, device="cuda")[:, 4:], E),
            ("cache", lambda t: t[:, :12].contiguous(), E), ("cache", lambda t: t[:, ::2], ValueError),
            ("cache", lambda t: t[None], ValueError), ("slot_mapping", lambda t: t.int(), TypeError),
            ("positions", lambda t: t.long(), TypeError), ("phases", lambda t: t[:16], ValueError),
            ("phases", lambda t: None, TypeError), ("weight", lambda t: t.half(), TypeError),
            ("weight", lambda t: t[:64], ValueError), ("q_out", lambda t: t[:2], ValueError),
            ("q_out", lambda t: t[:1].expand(3, 4, 64), E),
            ("eps", lambda t: -1.0, E), ("rope_scale", lambda t: float("inf"), E)]),
        (pkv.gather_latent, gather, [
            ("rows", lambda t: t[:, :256], ValueError), ("rows", lambda t: t.float(), TypeError),
            ("rows", lambda t: t.cpu(), ValueError), ("cache", lambda t: t.bfloat16(), TypeError),
            ("key_start", lambda t: t[:2], ValueError), ("key_start", lambda t: t.long(), TypeError),
            ("block_tables", lambda t: t[0], ValueError),
            ("rows", lambda t: gather["cache"].view(-1, 320)[:9], E)]),
        (pkv.latent_attention_prefill, prompt, [
            ("q", lambda t: t[..., :128], ValueError), ("q", lambda t: t.bfloat16(), TypeError),
            ("k", lambda t: t[:, :2], ValueError), ("k", lambda t: wide(t)[..., ::2], ValueError),
            ("v", lambda t: t[:5], ValueError), ("v", lambda t: t.cpu(), ValueError),
            ("k_rope", lambda t: t[:5], ValueError), ("k_rope", lambda t: t.float(), TypeError),
            ("out", lambda t: t.transpose(0, 1), ValueError), ("out", lambda t: t[..., :64], ValueError),
            ("query_start", lambda t: t[:2], ValueError), ("key_start", lambda t: t.long(), TypeError),
            ("scale", lambda t: float("nan"), E), ("max_query_len", lambda t: -1, E),
            ("max_key_len", lambda t: 1 << 40, ValueError), ("max_key_len", lambda t: -2, E),
            ("k", lambda t: t[:1].expand(7, 4, 128), E),
            ("out", lambda t: prompt["q"].view(-1)[:t.numel()].view(t.shape), E)]),
        (pkv.latent_attention_decode, decode, [
            ("out", lambda t: t[..., :128].contiguous(), E), ("out", lambda t: t[:2], ValueError),
            ("q", lambda t: t.transpose(0, 1), ValueError), ("q", lambda t: t.float(), TypeError),
            ("cache", lambda t: t[..., :256], ValueError), ("cache", lambda t: t.bfloat16(), TypeError),
            ("block_tables", lambda t: t.long(), TypeError), ("block_tables", lambda t: t[:1], ValueError),
            ("context_lens", lambda t: t[:1], ValueError), ("query_start", lambda t: t[:2], ValueError),
            ("query_start", lambda t: None, ValueError), ("ancestors", lambda t: t.int(), TypeError),
            ("ancestors", lambda t: t[:2], ValueError), ("max_query_len", lambda t: 65, E),
            ("max_query_len", lambda t: -1, E), ("scale", lambda t: float("inf"), E),
            ("scale", lambda t: "x", TypeError),
            ("workspace", lambda t: torch.empty(64, dtype=torch.uint8, device="cuda"), E),
            ("out", lambda t: decode["cache"].view(-1)[:t.numel()].view(t.shape), E)]),
    ]
    for fn, base, bad in cases:
        for name, change, error in bad:
            with pytest.raises(error):
                fn(**dict(base, **{name: change(base.get(name))}))
    # q_out beside q in one buffer, but not the same rows
    both = torch.zeros(3, 4, 128, dtype=torch.float16, device="cuda")
    with pytest.raises(E):
        pkv.latent_norm_rope_and_cache(**dict(write, q=both[..., :64], q_out=both[..., 64:]))
    torch.cuda.synchronize()
    assert pkv.get_device_error() == 0


def test_empty_batches_launch_nothing(pkv):
    import torch
    write, gather, prompt, decode = args(torch)
    e = lambda t: t[:0]  # noqa: E731
    pkv.latent_norm_rope_and_cache(**dict(write, **{n: e(write[n]) for n in (
        "q_out", "q", "latent", "k_rope", "slot_mapping", "positions")}))
    pkv.gather_latent(**dict(gather, rows=e(gather["rows"])))
    pkv.latent_attention_prefill(**dict(prompt, out=e(prompt["out"]), q=e(prompt["q"])))
    pkv.latent_attention_decode(**dict(decode, out=e(decode["out"]), q=e(decode["q"]),
                                       ancestors=e(decode["ancestors"])))
    # sequences without rows
    zero = torch.zeros(3, dtype=torch.int32, device="cuda")
    pkv.latent_attention_prefill(**dict(prompt, query_start=zero))
    pkv.latent_attention_decode(**dict(decode, query_start=zero))
    torch.cuda.synchronize()
    assert pkv.get_device_error() == 0


def test_one_head_and_one_token_of_any_stride(pkv):
    """Strides that lead nowhere are not looked at."""
    import torch
    write, _, prompt, _ = args(torch)
    q = torch.randn(1, 1, 70, device="cuda").half()[..., :64]
    one = dict(write, q=q, q_out=torch.empty(1, 1, 64, dtype=torch.half, device="cuda"),
               latent=write["latent"][:1], k_rope=write["k_rope"][:1],
               slot_mapping=write["slot_mapping"][:1], positions=write["positions"][:1],
               phases=pkv.rope_phases(pkv.rope_inv_freq(64)[0]))
    assert torch.equal(pkv.latent_norm_rope_and_cache(**one), q)
    k = torch.randn(1, 1, 132, device="cuda").half()[..., :128]
    z = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    out = torch.empty(1, 1, 128, dtype=torch.half, device="cuda")
    pkv.latent_attention_prefill(out, torch.randn(1, 1, 192, device="cuda").half(), k,
                                 prompt["k_rope"][:1], k, z, z, 0.1, 1, 1)
    assert torch.equal(out, k) and pkv.get_device_error() == 0
