"""The latent-attention operators together, as a serving step uses them: a prompt written
and attended in the expanded form, a chunk behind its gathered prefix, single tokens and a
drafted tree in the absorbed form; what they refuse; other streams; far places of a pool."""
import numpy as np
import pytest

from latent_helpers import P, check_decode, check_prefill, decode_case, on_device, prefill_case, run_decode

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_05_gb300 import build
    build.build()
    import paged_kv_cache_05_gb300 as m
    return m


class Layer:
    """Random projections of one attention layer, fp64 definitions beside the operators."""

    def __init__(self, torch, H, R, N, dtype):
        g = torch.Generator(device="cuda").manual_seed(H + R)
        r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.H, self.R, self.N, self.dt = H, R, N, dtype
        self.up_k = (r(H, N, R) / R ** 0.5).to(dtype)          # k_h = up_k[h] c
        self.up_v = (r(H, N, R) / R ** 0.5).to(dtype)
        self.weight = 1 + 0.1 * r(R)
        self.scale = (N + P) ** -0.5

    def expand(self, rows):
        """Keys and values of cached rows, as halves of one tensor [T, H, 2 N]."""
        import torch
        c = rows[:, :self.R]
        return torch.cat((torch.einsum("tr,hnr->thn", c, self.up_k),
                          torch.einsum("tr,hnr->thn", c, self.up_v)), -1)

    def exact(self, q, rows, see):
        """fp64 outputs in the latent space [T, H, R] of turned queries [T, H, N + P]."""
        import torch
        q, rows = q.double(), rows.double()
        full = torch.cat((torch.einsum("thn,hnr->thr", q[..., :self.N], self.up_k.double()),
                          q[..., self.N:]), -1)
        z = torch.einsum("thw,sw->ths", full, rows) * self.scale
        z = z.masked_fill(~see[:, None], -float("inf"))
        return torch.einsum("ths,sr->thr", torch.softmax(z, -1), rows[:, :self.R])


@pytest.mark.parametrize("H,R,N,B", [(16, 512, 128, 16), (5, 256, 64, 32)])
def test_prompt_chunk_token_tree(pkv, H, R, N, B):
    """150 tokens, a chunk of 70, a token, a tree of 6: every output against the definition
    over the rows that the cache then holds."""
    import torch
    dt = torch.bfloat16
    layer = Layer(torch, H, R, N, dt)
    g = torch.Generator(device="cuda").manual_seed(1)
    freq, rscale = pkv.rope_inv_freq(P, 10000.0)
    phases = pkv.rope_phases(freq)
    nb = 20
    cache = torch.full((nb, B, R + P), float("nan"), dtype=dt, device="cuda")
    bm = pkv.BlockManager(nb, B, 3)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    have = 0
    tree = [0b1, 0b11, 0b101, 0b1011, 0b10000, 0b110000]
    for n, kind in ((150, "prompt"), (70, "prompt"), (1, "token"), (6, "tree")):
        if have == 0:
            slots = bm.add_sequence(0, n)
        else:
            slots = np.array([bm.append_slot(0)[0] for _ in range(n)])
        tables, lens = bm.export([0], nb)
        down = (torch.randn(n, R + P, generator=g, device="cuda")).to(dt)
        q = (torch.randn(n, H, N + P, generator=g, device="cuda")).to(dt)
        pos = torch.arange(have, have + n, dtype=torch.int32, device="cuda")
        # rotary parts turned in place
        pkv.latent_norm_rope_and_cache(q[..., N:], q[..., N:], down[:, :R], down[:, R:], cache,
                                       torch.from_numpy(slots).cuda(), pos, phases,
                                       weight=layer.weight, rope_scale=rscale)
        have += n
        assert int(lens[0]) == have
        bt = torch.from_numpy(tables).cuda()
        rows = torch.empty(have, R + P, dtype=dt, device="cuda")
        pkv.gather_latent(rows, cache, bt, i32([0, have]))
        assert torch.isfinite(rows).all()
        t = torch.arange(have, device="cuda")
        see = t[None] <= (have - n + torch.arange(n, device="cuda"))[:, None]
        if kind == "tree":
            see = torch.stack([(t < have - n) | torch.tensor(
                [bool(t_ >= have - n and b >> (t_ - have + n) & 1) for t_ in range(have)],
                device="cuda") for b in tree])
        want = layer.exact(q, rows, see)
        if kind == "prompt":
            up = layer.expand(rows)
            out = torch.empty(n, H, N, dtype=dt, device="cuda")
            pkv.latent_attention_prefill(out, q, up[..., :N], rows[:, R:], up[..., N:], i32([0, n]),
                                         i32([0, have]), layer.scale, n, have)
            want = torch.einsum("thr,hnr->thn", want, layer.up_v.double())
            # keys and values rounded to the storage type, then weights and output
            assert (out.double() - want).abs().max() <= 0.05 * want.abs().max()
            assert (out.double() - want).norm() <= 0.01 * want.norm()
        else:
            full = torch.empty(n, H, R + P, dtype=dt, device="cuda")
            full[..., :R] = torch.einsum("thn,hnr->thr", q[..., :N], layer.up_k)
            full[..., R:] = q[..., N:]
            out = torch.empty(n, H, R, dtype=dt, device="cuda")
            pkv.latent_attention_decode(
                out, full, cache, bt, i32([have]), layer.scale, query_start=i32([0, n]),
                max_query_len=n,
                ancestors=torch.tensor(tree, device="cuda") if kind == "tree" else None)
            assert (out.double() - want).abs().max() <= 0.05 * want.abs().max()
            assert (out.double() - want).norm() <= 0.01 * want.norm()
        assert pkv.get_device_error() == 0


def test_more_sequences_than_threads(pkv):
    rs = np.random.RandomState(1)
    c = decode_case(rs, 3, 256, 8, [1] * 701, [int(x) for x in rs.randint(0, 40, 701)], "f16")
    check_decode(pkv, c, 0.07)
    new = [int(x) for x in rs.randint(0, 4, 900)]
    c = prefill_case(rs, 1, 64, new, [n + int(rs.randint(0, 9)) if n else 0 for n in new], "bf16")
    check_prefill(pkv, c, 0.07)


@pytest.mark.parametrize("scale", [-0.07, 0.0])
def test_negative_and_zero_scale(pkv, scale):
    rs = np.random.RandomState(2)
    check_decode(pkv, decode_case(rs, 16, 256, 16, [1, 5], [300, 90], "f16"), scale)
    check_prefill(pkv, prefill_case(rs, 2, 128, [130, 9], [130, 700], "bf16"), scale)


def test_on_another_stream_and_own_workspace(pkv):
    """Every call takes a stream; workspaces of the call's own are that stream's memory."""
    import torch
    rs = np.random.RandomState(3)
    c = decode_case(rs, 16, 512, 16, [1, 1], [1500, 200], "bf16")
    d = on_device(c)
    want = run_decode(pkv, c, 0.07, d)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(8):
        with torch.cuda.stream(side):
            junk = torch.full((64 << 20,), 255, dtype=torch.uint8, device="cuda")
        got = run_decode(pkv, c, 0.07, d, stream=side)
        del junk
        torch.cuda.synchronize()
        assert torch.equal(got, want)
    z = lambda *s: torch.randn(*s, device="cuda").half()  # noqa: E731
    cache, rows = z(4, 16, 320), z(40, 320)
    table = torch.tensor([[2, 0, 3]], dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    pkv.gather_latent(rows, cache, table, torch.tensor([0, 40], dtype=torch.int32, device="cuda"),
                      stream=side)
    torch.cuda.synchronize()
    assert torch.equal(rows, cache[[2, 0, 3]].reshape(-1, 320)[:40])


def test_captured_write_and_gather(pkv):
    import torch
    q, down = torch.randn(5, 2, P, device="cuda").half(), torch.randn(5, 256 + P, device="cuda").half()
    cache = torch.zeros(2, 8, 256 + P, dtype=torch.half, device="cuda")
    rows = torch.empty(5, 256 + P, dtype=torch.half, device="cuda")
    slots, pos = torch.arange(8, 13, device="cuda"), torch.arange(5, dtype=torch.int32, device="cuda")
    phases = pkv.rope_phases(pkv.rope_inv_freq(P)[0])
    out = torch.empty_like(q)
    table = torch.tensor([[1, 0]], dtype=torch.int32, device="cuda")
    ks = torch.tensor([0, 5], dtype=torch.int32, device="cuda")

    def step():
        pkv.latent_norm_rope_and_cache(out, q, down[:, :256], down[:, 256:], cache, slots, pos, phases)
        pkv.gather_latent(rows, cache, table, ks)

    g = torch.cuda.CUDAGraph()
    step()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        step()
    q.mul_(2)
    down.mul_(-1)
    g.replay()
    got = out.clone(), rows.clone()
    step()
    torch.cuda.synchronize()
    assert torch.equal(got[0], out) and torch.equal(got[1], rows)
    assert torch.equal(rows[:, :256], down[:, :256])


def test_far_places(pkv):
    """Blocks beyond 2^31 elements of a pool: written, gathered and attended."""
    import torch
    R, B, nb = 512, 64, 60000                      # 2.2e9 elements
    cache = torch.empty(nb, B, R + P, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(4)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    n = 150
    blocks = torch.tensor([nb - 1, 3, nb - 2], dtype=torch.int32, device="cuda")
    t = torch.arange(n, device="cuda")
    slots = blocks[t // B].long() * B + t % B
    down, q = r(n, R + P), r(n, 4, P)
    phases = pkv.rope_phases(pkv.rope_inv_freq(P)[0])
    pkv.latent_norm_rope_and_cache(q, q, down[:, :R], down[:, R:], cache, slots, torch.zeros_like(t).int(),
                                   phases)         # position 0 turns nothing
    rows = torch.empty(n, R + P, dtype=torch.bfloat16, device="cuda")
    pkv.gather_latent(rows, cache, blocks[None], torch.tensor([0, n], dtype=torch.int32, device="cuda"))
    assert torch.equal(rows, down)
    qa, out = r(1, 16, R + P), torch.empty(1, 16, R, dtype=torch.bfloat16, device="cuda")
    pkv.latent_attention_decode(out, qa, cache, blocks[None],
                                torch.tensor([n], dtype=torch.int32, device="cuda"), 0.05)
    want = torch.softmax(0.05 * qa[0].double() @ rows.double().T, -1) @ rows[:, :R].double()
    # the weights' rounding and the output's: half a step each, the weights' twice
    size = torch.softmax(0.05 * qa[0].double() @ rows.double().T, -1) @ rows[:, :R].double().abs()
    assert ((out[0].double() - want).abs() <= 2.0 ** -8 * (2 * size + want.abs()) + 1e-3 * size).all()
    assert pkv.get_device_error() == 0
