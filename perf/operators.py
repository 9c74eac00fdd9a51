"""The grouped-head serving step over the paged cache, as measured cases.

Three operators that follow one another in a model whose query heads share
key/value heads: the new tokens' query/key norm, rotation and cache write; the
attention of a prompt's tokens over the cache; the attention of one new token
per sequence over the cache.

``run`` computes a case in its plain form (torch products, sums, exp and
indexing in 32 bits, angles in 64) while ``own`` is false, and calls this
repository's operators when it is true.  ``exact`` is the same from the
definitions in 64 bits.
"""
import math
import random

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------- cases
def listed():
    return [
        # --- norm + rotation + cache write
        # one sequence's decode step: a single token, latency only
        _rope("write one token", T=1, H=32, HK=8, D=128, rot=128, B=16, dtype="bf16", norm=True,
              interleaved=False, far=32768),
        # a decode step of 64 sequences, 40 query heads, no norm, interleaved pairs
        _rope("write 64 tokens", T=64, H=40, HK=8, D=128, rot=128, B=16, dtype="f16", norm=False,
              interleaved=True, far=4096),
        # a ragged prompt batch of a small-headed model, half of each head rotated
        _rope("write 4099 tokens", T=4099, H=24, HK=6, D=64, rot=32, B=32, dtype="f16", norm=True,
              interleaved=False, far=8192),
        # a large prompt batch at positions far into a scaled long context
        _rope("write 16384 tokens", T=16384, H=32, HK=8, D=128, rot=128, B=16, dtype="bf16",
              norm=True, interleaved=False, far=131072),
        # --- one new token per sequence
        # a single short conversation: latency
        _decode("decode one sequence", S=1, lo=500, hi=500, H=32, HK=8, D=128, B=16, dtype="bf16",
                cap=0.0, window=0, slopes=False),
        # a serving batch of mixed lengths with capped scores
        _decode("decode 64 capped", S=64, lo=1, hi=2048, H=40, HK=8, D=128, B=16, dtype="f16",
                cap=30.0, window=0, slopes=False),
        # one shared key/value head, a sliding window and a distance bias
        _decode("decode 33 windowed", S=33, lo=17, hi=8191, H=16, HK=1, D=64, B=64, dtype="bf16",
                cap=0.0, window=1000, slopes=True),
        # long documents
        _decode("decode 8 long", S=8, lo=8192, hi=32768, H=32, HK=8, D=128, B=16, dtype="bf16",
                cap=0.0, window=0, slopes=False),
        # --- prompts
        # one short prompt: latency
        _prompt("prompt of 61", S=1, lo=61, hi=61, past=0, H=32, HK=8, D=128, B=16, dtype="bf16",
                cap=0.0, window=0, slopes=False),
        # a batch of ragged prompts with a distance bias
        _prompt("prompts biased", S=8, lo=100, hi=1100, past=0, H=24, HK=6, D=64, B=32, dtype="f16",
                cap=0.0, window=0, slopes=True),
        # prompts continued after a cached prefix, capped scores and a sliding window
        _prompt("chunks windowed", S=4, lo=301, hi=1024, past=5000, H=16, HK=4, D=128, B=16,
                dtype="bf16", cap=50.0, window=1024, slopes=False),
        # whole long prompts
        _prompt("prompts of 2048", S=4, lo=1900, hi=2048, past=0, H=32, HK=8, D=128, B=16,
                dtype="f16", cap=0.0, window=0, slopes=False),
    ]


def _rope(name, **kw):
    return dict(name=name, op="write", **kw)


def _decode(name, **kw):
    return dict(name=name, op="decode", **kw)


def _prompt(name, **kw):
    return dict(name=name, op="prompt", **kw)


def draw(rng):
    most = {}
    for c in listed():
        w = work(c)
        b, f = most.get(c["op"], (0, 0))
        most[c["op"]] = (max(b, w["bytes"]), max(f, w["flops"]))
    log = lambda lo, hi: max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))  # noqa: E731
    while True:
        op = rng.choice(("write", "decode", "prompt"))
        c = dict(op=op, HK=rng.choice((1, 2, 3, 4, 6, 8)), D=rng.choice((64, 128)),
                 B=rng.choice((8, 16, 32, 64)), dtype=rng.choice(("f16", "bf16")))
        c["H"] = c["HK"] * rng.choice((1, 2, 3, 4, 5, 7, 8, 12, 16))
        if op == "write":
            c.update(T=log(1, 16384), rot=8 * rng.randint(1, c["D"] // 8),
                     norm=rng.random() < 0.5, interleaved=rng.random() < 0.5,
                     far=log(1000, 131072))
        else:
            hi = log(1, 32768) if op == "decode" else log(1, 2048)
            c.update(S=log(1, 64) if op == "decode" else log(1, 8), hi=hi, lo=log(1, hi),
                     cap=rng.choice((0.0, 20.0, 50.0)), slopes=rng.random() < 0.3,
                     window=log(1, 8192) if rng.random() < 0.3 else 0)
            if op == "prompt":
                c["past"] = log(1, 6000) if rng.random() < 0.5 else 0
        w = work(c)
        padded = 1 if op == "write" else c["S"] * (c["hi"] + c.get("past", 0)) * c["HK"] * c["D"]
        scores = c["S"] * c["H"] * c["hi"] * (c["hi"] + c["past"]) if op == "prompt" else 1
        if (w["bytes"] <= most[op][0] and w["flops"] <= most[op][1] and padded <= 8 * 32768 * 1024
                and scores <= 4 * 32 * 2048 * 2048):
            return c


def _lengths(case):
    """Per sequence: (new tokens, tokens attended), the same for every seed."""
    r = random.Random(977 * case["S"] + 31 * case["hi"] + case["lo"])
    new = [r.randint(case["lo"], case["hi"]) for _ in range(case["S"])]
    if case["op"] == "decode":
        return [1] * len(new), new
    past = [r.randint(case["past"] // 2, case["past"]) for _ in new]
    return new, [n + p for n, p in zip(new, past)]


def work(case):
    H, HK, D = case["H"], case["HK"], case["D"]
    if case["op"] == "write":
        T = case["T"]
        # q, k, v in; q and the cache rows out; a position and a slot per token
        return {"bytes": T * (2 * (H + 2 * HK) * D * 2 + 12) + 8 * case["rot"] // 2,
                "flops": T * (H + HK) * D * (6 if case["norm"] else 3)}
    new, ctx = _lengths(case)
    w = case["window"]
    pairs = tokens = 0
    for n, c in zip(new, ctx):
        first = c - n                                  # position of the first query
        if w <= 0:
            pairs += n * (2 * first + n + 1) // 2
            tokens += c
        else:
            full = max(0, c - max(first, w - 1))       # queries that see a whole window
            part = n - full                            # positions first .. first + part - 1
            pairs += full * w + part * (2 * first + part + 1) // 2
            tokens += c - max(0, first + 1 - w)
    rows = sum(new)
    return {"bytes": 2 * tokens * HK * D * 2 + 2 * rows * H * D * 2
            + 4 * sum(-(-c // case["B"]) for c in ctx) + 8 * len(ctx),
            "flops": 4 * pairs * H * D}


# ------------------------------------------------------------------- inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, dtype, times=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * times).to(dtype)


def prepare(case, seed):
    g = _generator(seed)
    return _prepare_write(case, g) if case["op"] == "write" else _prepare_attention(case, g)


def _prepare_write(case, g):
    T, H, HK, D, B, rot = (case[k] for k in ("T", "H", "HK", "D", "B", "rot"))
    dt = DTYPES[case["dtype"]]
    # the projection's output: queries, keys and values of a token side by side
    qkv = _normal(g, (T, (H + 2 * HK) * D), dt, 1.5)
    nb = -(-T // B) + 3
    inv_freq = 500000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    # a pair's angle per position, in 2^-64 turns
    phases = [round(float(f) / (2 * math.pi) * 2.0 ** 64) for f in inv_freq]
    phases = [p - (1 << 64) if p >= 1 << 63 else p for p in phases]
    st = dict(case=case,
              q=qkv[:, :H * D].view(T, H, D), k=qkv[:, H * D:(H + HK) * D].view(T, HK, D),
              v=qkv[:, (H + HK) * D:].view(T, HK, D),
              k_cache=_normal(g, (nb, HK, B, D), dt), v_cache=_normal(g, (nb, HK, B, D), dt),
              slots=torch.randperm(nb * B, generator=g, device="cuda")[:T],
              positions=torch.randint(0, case["far"], (T,), generator=g, device="cuda",
                                      dtype=torch.int32),
              inv_freq=inv_freq.cuda(), phases=torch.tensor(phases, device="cuda"),
              q_weight=None, k_weight=None, eps=1e-6, rope_scale=1.0 if rot == D else 1.125,
              q_out=torch.empty((T, H, D), dtype=dt, device="cuda"))
    if case["norm"]:
        st["q_weight"] = 1 + 0.2 * torch.randn(D, generator=g, device="cuda")
        st["k_weight"] = 1 + 0.2 * torch.randn(D, generator=g, device="cuda")
    return st


def _prepare_attention(case, g):
    H, HK, D, B, S = (case[k] for k in ("H", "HK", "D", "B", "S"))
    dt = DTYPES[case["dtype"]]
    new, ctx = _lengths(case)
    counts = [-(-c // B) for c in ctx]
    nb, width = sum(counts) + 5, max(counts)
    blocks = torch.randperm(nb, generator=g, device="cuda").to(torch.int32)
    start = torch.tensor([0] + counts[:-1], device="cuda").cumsum(0)
    col = torch.arange(width, device="cuda")
    held = col[None] < torch.tensor(counts, device="cuda")[:, None]
    tables = torch.where(held, blocks[(start[:, None] + col).clamp(max=nb - 1)], -1)
    rows = sum(new)
    # capped scores matter where they are large
    q = _normal(g, (rows, H, D), dt, 6.0 if case["cap"] else 1.0)
    slopes = None
    if case["slopes"]:
        slopes = 2.0 ** (-8.0 * torch.arange(1, H + 1, device="cuda", dtype=torch.float32) / H)
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    return dict(case=case, q=q, out=torch.empty_like(q),
                k_cache=_normal(g, (nb, HK, B, D), dt), v_cache=_normal(g, (nb, HK, B, D), dt),
                tables=tables.to(torch.int32).contiguous(),
                context_lens=torch.tensor(ctx, dtype=torch.int32, device="cuda"),
                query_start=torch.tensor(starts, dtype=torch.int32, device="cuda"),
                max_query_len=max(new), scale=1.0 / math.sqrt(D), slopes=slopes, workspace=None)


# ------------------------------------------------------------------- run
def run(state):
    if own:
        return _run_own(state)
    return _plain_write(state) if state["case"]["op"] == "write" else _plain_attention(state)


def _run_own(st):
    import paged_kv_cache_05_gb300 as pkv
    c = st["case"]
    if c["op"] == "write":
        pkv.norm_rope_and_cache(st["q_out"], st["q"], st["k"], st["v"], st["k_cache"],
                                st["v_cache"], st["slots"], st["positions"], st["phases"],
                                q_weight=st["q_weight"], k_weight=st["k_weight"], eps=st["eps"],
                                rope_scale=st["rope_scale"], interleaved=c["interleaved"])
        return st["q_out"], st["k_cache"], st["v_cache"]
    if c["op"] == "decode":
        if st["workspace"] is None:
            st["workspace"] = pkv.alloc_grouped_workspace(c["S"], c["H"], c["HK"], c["D"], c["B"],
                                                          st["tables"].shape[1])
        return pkv.paged_attention_decode_grouped(
            st["out"], st["q"], st["k_cache"], st["v_cache"], st["tables"], st["context_lens"],
            st["scale"], softcap=c["cap"], window=c["window"], slopes=st["slopes"],
            workspace=st["workspace"])
    return pkv.paged_attention_prefill_grouped(
        st["out"], st["q"], st["k_cache"], st["v_cache"], st["tables"], st["context_lens"],
        st["query_start"], st["scale"], st["max_query_len"], softcap=c["cap"],
        window=c["window"], slopes=st["slopes"])


def _plain_write(st):
    c = st["case"]
    half = c["rot"] // 2
    angle = st["positions"].double()[:, None, None] * st["inv_freq"]
    cos, sin = (f(angle).float() * st["rope_scale"] for f in (torch.cos, torch.sin))

    def turned(x, weight):
        x = x.float()
        if weight is not None:
            x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + st["eps"]) * weight
        r, rest = x[..., :c["rot"]], x[..., c["rot"]:]
        if c["interleaved"]:
            a, b = r[..., 0::2], r[..., 1::2]
            r = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
        else:
            a, b = r[..., :half], r[..., half:]
            r = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
        return torch.cat((r, rest), -1).to(st["q"].dtype)

    st["q_out"].copy_(turned(st["q"], st["q_weight"]))
    block, offset = st["slots"] // c["B"], st["slots"] % c["B"]
    st["k_cache"][block, :, offset] = turned(st["k"], st["k_weight"])
    st["v_cache"][block, :, offset] = st["v"]
    return st["q_out"], st["k_cache"], st["v_cache"]


def _plain_attention(st):
    c = st["case"]
    S, H, HK, D = c["S"], c["H"], c["HK"], c["D"]
    G, dev = H // HK, st["q"].device
    ctx, starts = st["context_lens"].long(), st["query_start"].long()
    new = starts[1:] - starts[:-1]
    blocks = st["tables"].long().clamp(min=0)
    # every sequence's keys and values, padded to the longest: [S, HK, tokens, D]
    k = st["k_cache"][blocks].transpose(1, 2).flatten(2, 3).float()
    v = st["v_cache"][blocks].transpose(1, 2).flatten(2, 3).float()
    t = torch.arange(k.shape[2], device=dev)
    i = torch.arange(st["max_query_len"], device=dev)
    row = (starts[:-1, None] + i).clamp(max=st["q"].shape[0] - 1)
    q = st["q"][row].float().view(S, -1, HK, G, D).permute(0, 2, 3, 1, 4)     # [S, HK, G, new, D]
    p = (ctx - new)[:, None] + i                                              # query positions
    z = torch.matmul(q.flatten(2, 3), k.transpose(-1, -2)).view(S, HK, G, -1, t.shape[0])
    z = z * st["scale"]
    if c["cap"]:
        z = torch.tanh(z / c["cap"]) * c["cap"]
    if st["slopes"] is not None:
        z = z + st["slopes"].view(HK, G, 1, 1) * (t - p[:, None, None, :, None])
    seen = t <= p[:, :, None]
    if c["window"]:
        seen = seen & (t > p[:, :, None] - c["window"])
    z = z.masked_fill(~seen[:, None, None], -math.inf)
    e = torch.exp(z - z.amax(-1, keepdim=True))
    o = torch.matmul(e.flatten(2, 3), v).view(S, HK, G, -1, D) / e.sum(-1)[..., None]
    o = o.permute(0, 3, 1, 2, 4).reshape(S, -1, H, D)
    flat = torch.arange(st["q"].shape[0], device=dev)
    seq = torch.searchsorted(starts[1:].contiguous(), flat, right=True)
    st["out"].copy_(o[seq, flat - starts[seq]])
    return st["out"]


# ------------------------------------------------------------------- 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    return _exact_write(st) if case["op"] == "write" else _exact_attention(st)


def _exact_write(st):
    c = st["case"]
    D, rot, B = c["D"], c["rot"], c["B"]
    # each pair as a complex number, multiplied by the unit number of its angle
    unit = torch.polar(torch.full_like(st["inv_freq"], st["rope_scale"])[None],
                       st["positions"].double()[:, None] * st["inv_freq"][None])[:, None]
    first = torch.arange(0, rot, 2) if c["interleaved"] else torch.arange(rot // 2)
    second = first + (1 if c["interleaved"] else rot // 2)

    def turned(x, weight):
        x = x.double()
        if weight is not None:
            x = x * (x.pow(2).sum(-1, keepdim=True) / D + st["eps"]).rsqrt() * weight.double()
        y = x.clone()
        z = torch.complex(x[..., first], x[..., second]) * unit
        y[..., first], y[..., second] = z.real, z.imag
        return y

    k_cache, v_cache = st["k_cache"].double(), st["v_cache"].double()
    for pool, new in ((k_cache, turned(st["k"], st["k_weight"])), (v_cache, st["v"].double())):
        for h in range(c["HK"]):
            flat = pool[:, h].reshape(-1, D)
            flat[st["slots"]] = new[:, h]
            pool[:, h] = flat.view(-1, B, D)
    return turned(st["q"], st["q_weight"]), k_cache, v_cache


def _exact_attention(st):
    c = st["case"]
    H, HK, B, D = c["H"], c["HK"], c["B"], c["D"]
    starts, ctx = st["query_start"].tolist(), st["context_lens"].tolist()
    out = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
    for s, n in enumerate(ctx):
        token = torch.arange(n, device="cuda")
        block = st["tables"][s].long()[token // B]
        rows = slice(starts[s], starts[s + 1])
        pos = torch.arange(n - (starts[s + 1] - starts[s]), n, device="cuda")
        ahead = pos[:, None] - token[None]
        hidden = ahead < 0
        if c["window"]:
            hidden |= ahead >= c["window"]
        for h in range(H):
            k = st["k_cache"][block, h * HK // H, token % B].double()
            v = st["v_cache"][block, h * HK // H, token % B].double()
            z = st["q"][rows, h].double() @ k.T * st["scale"]
            if c["cap"]:
                z = c["cap"] * torch.tanh(z / c["cap"])
            if st["slopes"] is not None:
                z -= st["slopes"][h].double() * ahead
            out[rows, h] = torch.softmax(z.masked_fill(hidden, -math.inf), -1) @ v
    return out
