"""The serving step of a model with latent attention, as measured cases.

Such a model keeps one shared row a token in its cache: a latent vector, from
which every head's key and value would be formed, and one rotated key part that
all heads share.  Four operators that follow one another:

    write   the new tokens' latent norm, rotation of the shared key part and of the
            queries' rotary parts, and the write of the cache rows
    gather  a sequence's cached rows as contiguous rows, from which a chunk of a
            prompt forms the keys and values of the tokens before it
    prompt  attention in the expanded form: keys of a per-head part and the shared
            rotated part, values per head, causal, ragged sequences
    decode  attention in the absorbed form: queries taken into the latent space, the
            cache rows are keys and (their latent part) values of every head; one new
            token a sequence, several, or a tree of drafted ones

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
P = 64                                  # the rotated part of a key or query


# ------------------------------------------------------------------- cases
def listed():
    return [
        # --- norm + rotation + cache write
        # one sequence's decode step: a single token, latency only
        _write("write one token", T=1, H=16, R=512, B=16, dtype="bf16", norm=True,
               interleaved=True, far=32768),
        # a decode step of 64 sequences with many query heads
        _write("write 64 tokens", T=64, H=128, R=512, B=64, dtype="bf16", norm=True,
               interleaved=True, far=8192),
        # a ragged prompt batch, halves of the rotated part as pairs, no norm
        _write("write 16001 tokens", T=16001, H=32, R=256, B=32, dtype="f16", norm=False,
               interleaved=False, far=131072),
        # --- cached rows as contiguous ones
        # one short conversation's prefix
        _gather("gather one prefix", S=1, lo=700, hi=700, R=512, B=16, dtype="bf16"),
        # the prefixes of a batch of long documents
        _gather("gather 8 prefixes", S=8, lo=4097, hi=16384, R=512, B=16, dtype="bf16"),
        # --- prompts, expanded
        # one short prompt: latency
        _prompt("prompt of 61", S=1, lo=61, hi=61, past=0, H=16, N=128, dtype="bf16"),
        # chunks of long prompts behind a gathered prefix, narrow heads
        _prompt("chunks", S=4, lo=301, hi=1024, past=5000, H=16, N=64, dtype="f16"),
        # whole long prompts
        _prompt("prompts of 2048", S=4, lo=1900, hi=2048, past=0, H=32, N=128, dtype="bf16"),
        # --- new tokens over the cache, absorbed
        # a single short conversation: latency
        _decode("decode one sequence", S=1, lo=500, hi=500, new=1, tree=False, H=16, R=512, B=16,
                dtype="bf16"),
        # a serving batch of mixed lengths with many heads
        _decode("decode 64", S=64, lo=1, hi=2048, new=1, tree=False, H=128, R=512, B=64,
                dtype="bf16"),
        # trees of drafted tokens verified
        _decode("decode 33 trees", S=33, lo=77, hi=4095, new=13, tree=True, H=20, R=256, B=32,
                dtype="f16"),
        # long documents
        _decode("decode 8 long", S=8, lo=8192, hi=32768, new=1, tree=False, H=16, R=512, B=16,
                dtype="bf16"),
    ]


def _write(name, **kw):
    return dict(name=name, op="write", **kw)


def _gather(name, **kw):
    return dict(name=name, op="gather", **kw)


def _prompt(name, **kw):
    return dict(name=name, op="prompt", **kw)


def _decode(name, **kw):
    return dict(name=name, op="decode", **kw)


def draw(rng):
    most = {}
    for c in listed():
        w = work(c)
        b, f = most.get(c["op"], (0, 0))
        most[c["op"]] = (max(b, w["bytes"]), max(f, w["flops"]))
    log = lambda lo, hi: max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))  # noqa: E731
    while True:
        op = rng.choice(("write", "gather", "prompt", "decode", "decode"))
        c = dict(op=op, dtype=rng.choice(("f16", "bf16")))
        padded = scores = 1
        if op != "prompt":
            c.update(R=rng.choice((256, 512)), B=rng.choice((8, 16, 32, 64)))
        if op != "gather":
            c["H"] = rng.choice((1, 3, 8, 16, 20, 32, 64, 128))
        if op == "write":
            c.update(T=log(1, 16384), norm=rng.random() < 0.7, interleaved=rng.random() < 0.5,
                     far=log(1000, 131072))
        elif op == "gather":
            hi = log(1, 32768)
            c.update(S=log(1, 64), hi=hi, lo=log(1, hi))
            padded = c["S"] * hi * (c["R"] + P)
        elif op == "prompt":
            hi = log(1, 2048)
            c.update(S=log(1, 8), hi=hi, lo=log(1, hi), N=rng.choice((64, 128)),
                     past=log(1, 6000) if rng.random() < 0.5 else 0)
            scores = c["S"] * c["H"] * hi * (hi + c["past"])
        else:
            hi = log(1, 32768)
            new = 1 if rng.random() < 0.5 else log(2, 64)
            c.update(S=log(1, 64), hi=max(hi, new), new=new, tree=new > 1 and rng.random() < 0.6)
            c["lo"] = log(new, c["hi"])
            padded = c["S"] * c["hi"] * (c["R"] + P)
            scores = c["S"] * c["hi"] * c["H"] * new
        w = work(c)
        if (w["bytes"] <= most[op][0] and w["flops"] <= most[op][1] and padded <= 8 * 32768 * 576
                and scores <= 4 * 32 * 2048 * 2048):
            return c


def _lengths(case):
    """Per sequence: (new tokens, tokens attended), the same for every seed."""
    r = random.Random(977 * case["S"] + 31 * case["hi"] + case["lo"])
    tokens = [r.randint(case["lo"], case["hi"]) for _ in range(case["S"])]
    if case["op"] == "gather":
        return [0] * len(tokens), tokens
    if case["op"] == "decode":
        return [r.randint(1, case["new"]) if case["tree"] else case["new"] for _ in tokens], tokens
    past = [r.randint(case["past"] // 2, case["past"]) for _ in tokens]
    return tokens, [n + p for n, p in zip(tokens, past)]


def work(case):
    if case["op"] == "write":
        T, H, W = case["T"], case["H"], case["R"] + P
        # latent and shared key part in, cache rows out; rotary parts of the queries in and out;
        # a position and a slot per token
        return {"bytes": T * (4 * W + 4 * H * P + 12) + 8 * P // 2,
                "flops": T * ((H + 1) * P * 3 + (4 * case["R"] if case["norm"] else 0))}
    new, ctx = _lengths(case)
    if case["op"] == "gather":
        rows = sum(ctx)
        return {"bytes": 4 * rows * (case["R"] + P) + 4 * sum(-(-c // case["B"]) for c in ctx),
                "flops": 0}
    H = case["H"]
    # a tree's rows see as many of the drafted tokens as a chain's at most
    pairs = sum(n * (2 * (c - n) + n + 1) // 2 for n, c in zip(new, ctx))
    if case["op"] == "prompt":
        N = case["N"]
        return {"bytes": 2 * sum(new) * H * (2 * N + P) + 2 * sum(ctx) * (2 * H * N + P)
                + 8 * len(ctx),
                "flops": 2 * pairs * H * (2 * N + P)}
    R, W = case["R"], case["R"] + P
    return {"bytes": 2 * sum(ctx) * W + 2 * sum(new) * H * (W + R)
            + 4 * sum(-(-c // case["B"]) for c in ctx) + 4 * len(ctx),
            "flops": 2 * pairs * H * (W + R)}


# ------------------------------------------------------------------- inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, dtype, times=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * times).to(dtype)


def _starts(counts):
    s = [0]
    for n in counts:
        s.append(s[-1] + n)
    return torch.tensor(s, dtype=torch.int32, device="cuda")


def _tables(g, ctx, B):
    """Block tables of sequences scattered through a pool, -1 past their ends; blocks in it."""
    counts = [-(-c // B) for c in ctx]
    nb, width = sum(counts) + 5, max(counts)
    blocks = torch.randperm(nb, generator=g, device="cuda").to(torch.int32)
    start = torch.tensor([0] + counts[:-1], device="cuda").cumsum(0)
    col = torch.arange(width, device="cuda")
    held = col[None] < torch.tensor(counts, device="cuda")[:, None]
    tables = torch.where(held, blocks[(start[:, None] + col).clamp(max=nb - 1)], -1)
    return tables.to(torch.int32).contiguous(), nb


def prepare(case, seed):
    g = _generator(seed)
    return {"write": _prepare_write, "gather": _prepare_gather, "prompt": _prepare_prompt,
            "decode": _prepare_decode}[case["op"]](case, g)


def _prepare_write(case, g):
    T, H, R, B = (case[k] for k in ("T", "H", "R", "B"))
    dt = DTYPES[case["dtype"]]
    down = _normal(g, (T, R + P), dt, 1.5)            # the joint down-projection's output
    query = _normal(g, (T, H, 128 + P), dt, 1.5)      # the query projection's
    nb = -(-T // B) + 3
    inv_freq = 500000.0 ** (-torch.arange(0, P, 2, dtype=torch.float64) / P)
    # a pair's angle per position, in 2^-64 turns
    phases = [round(float(f) / (2 * math.pi) * 2.0 ** 64) for f in inv_freq]
    phases = [p - (1 << 64) if p >= 1 << 63 else p for p in phases]
    # queries in the latent space beside their rotary parts, as the attention reads them
    absorbed = torch.zeros((T, H, R + P), dtype=dt, device="cuda")
    return dict(case=case, latent=down[:, :R], k_rope=down[:, R:], q=query[..., 128:],
                q_out=absorbed[..., R:], cache=_normal(g, (nb, B, R + P), dt),
                slots=torch.randperm(nb * B, generator=g, device="cuda")[:T],
                positions=torch.randint(0, case["far"], (T,), generator=g, device="cuda",
                                        dtype=torch.int32),
                inv_freq=inv_freq.cuda(), phases=torch.tensor(phases, device="cuda"),
                weight=(1 + 0.2 * torch.randn(R, generator=g, device="cuda")) if case["norm"]
                else None,
                eps=1e-6, rope_scale=1.0 if case["norm"] else 1.125)


def _prepare_gather(case, g):
    _, ctx = _lengths(case)
    tables, nb = _tables(g, ctx, case["B"])
    W, dt = case["R"] + P, DTYPES[case["dtype"]]
    return dict(case=case, cache=_normal(g, (nb, case["B"], W), dt), tables=tables,
                key_start=_starts(ctx),
                rows=torch.empty((sum(ctx), W), dtype=dt, device="cuda"))


def _prepare_prompt(case, g):
    H, N = case["H"], case["N"]
    dt = DTYPES[case["dtype"]]
    new, keys = _lengths(case)
    up = _normal(g, (sum(keys), H, 2 * N), dt)        # the up-projection's output: keys, values
    cached = _normal(g, (sum(keys), 256 + P), dt)     # gathered cache rows
    return dict(case=case, q=_normal(g, (sum(new), H, N + P), dt), k=up[..., :N], v=up[..., N:],
                k_rope=cached[:, 256:], out=torch.empty((sum(new), H, N), dtype=dt, device="cuda"),
                query_start=_starts(new), key_start=_starts(keys), max_query_len=max(new),
                max_key_len=max(keys), scale=1.0 / math.sqrt(N + P))


def _prepare_decode(case, g):
    H, R, B = case["H"], case["R"], case["B"]
    dt = DTYPES[case["dtype"]]
    new, ctx = _lengths(case)
    tables, nb = _tables(g, ctx, B)
    q = _normal(g, (sum(new), H, R + P), dt)
    ancestors = None
    if case["tree"]:
        # each drafted token hangs under an earlier one of its sequence, or under the cache
        r = random.Random(len(ctx) + case["hi"])
        bits = []
        for n in new:
            seen = []
            for j in range(n):
                parent = r.randint(-1, j - 1)
                seen.append((seen[parent] if parent >= 0 else 0) | 1 << j)
            bits += [b - (1 << 64) if b >= 1 << 63 else b for b in seen]
        ancestors = torch.tensor(bits, dtype=torch.int64, device="cuda")
    return dict(case=case, q=q, out=torch.empty((sum(new), H, R), dtype=dt, device="cuda"),
                cache=_normal(g, (nb, B, R + P), dt), tables=tables,
                context_lens=torch.tensor(ctx, dtype=torch.int32, device="cuda"),
                query_start=_starts(new), max_query_len=max(new), ancestors=ancestors,
                scale=1.0 / math.sqrt(128 + P), workspace=None)


# ------------------------------------------------------------------- run
def run(state):
    if own:
        return _run_own(state)
    return {"write": _plain_write, "gather": _plain_gather, "prompt": _plain_prompt,
            "decode": _plain_decode}[state["case"]["op"]](state)


def _run_own(st):
    import paged_kv_cache_05_gb300 as pkv
    c = st["case"]
    if c["op"] == "write":
        pkv.latent_norm_rope_and_cache(
            st["q_out"], st["q"], st["latent"], st["k_rope"], st["cache"], st["slots"],
            st["positions"], st["phases"], weight=st["weight"], eps=st["eps"],
            rope_scale=st["rope_scale"], interleaved=c["interleaved"])
        return st["q_out"], st["cache"]
    if c["op"] == "gather":
        return pkv.gather_latent(st["rows"], st["cache"], st["tables"], st["key_start"])
    if c["op"] == "prompt":
        return pkv.latent_attention_prefill(
            st["out"], st["q"], st["k"], st["k_rope"], st["v"], st["query_start"],
            st["key_start"], st["scale"], st["max_query_len"], st["max_key_len"])
    if st["workspace"] is None:
        st["workspace"] = pkv.alloc_latent_workspace(c["S"], c["H"], c["R"], st["max_query_len"])
    return pkv.latent_attention_decode(
        st["out"], st["q"], st["cache"], st["tables"], st["context_lens"], st["scale"],
        query_start=st["query_start"], max_query_len=st["max_query_len"],
        ancestors=st["ancestors"], workspace=st["workspace"])


def _plain_write(st):
    c = st["case"]
    angle = st["positions"].double()[:, None] * st["inv_freq"]
    cos, sin = (f(angle).float() * st["rope_scale"] for f in (torch.cos, torch.sin))

    def turned(x, cos, sin):
        x = x.float()
        if c["interleaved"]:
            a, b = x[..., 0::2], x[..., 1::2]
            x = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
        else:
            a, b = x[..., :P // 2], x[..., P // 2:]
            x = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
        return x.to(st["q"].dtype)

    st["q_out"].copy_(turned(st["q"], cos[:, None], sin[:, None]))
    x = st["latent"].float()
    if st["weight"] is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + st["eps"]) * st["weight"]
    block, offset = st["slots"] // c["B"], st["slots"] % c["B"]
    st["cache"][block, offset] = torch.cat((x.to(st["q"].dtype), turned(st["k_rope"], cos, sin)), -1)
    return st["q_out"], st["cache"]


def _plain_gather(st):
    B = st["case"]["B"]
    start = st["key_start"].long()
    row = torch.arange(st["rows"].shape[0], device="cuda")
    seq = torch.searchsorted(start[1:].contiguous(), row, right=True)
    t = row - start[seq]
    st["rows"].copy_(st["cache"][st["tables"][seq, t // B].long(), t % B])
    return st["rows"]


def _padded(x, start, most):
    """Ragged rows as [sequences, most, ...]; rows past a sequence's end are some other row."""
    i = start[:-1, None].long() + torch.arange(most, device=x.device)
    return x[i.clamp(max=x.shape[0] - 1)]


def _ragged(x, start, n):
    """And back: the first rows of each sequence, n in all."""
    flat = torch.arange(n, device=x.device)
    seq = torch.searchsorted(start[1:].long().contiguous(), flat, right=True)
    return x[seq, flat - start.long()[seq]]


def _plain_prompt(st):
    qs, ks = st["query_start"].long(), st["key_start"].long()
    nq, nk = qs[1:] - qs[:-1], ks[1:] - ks[:-1]
    H = st["case"]["H"]
    q = _padded(st["q"], qs, st["max_query_len"]).float().transpose(1, 2)       # [S, H, new, N+P]
    shared = st["k_rope"].float()[:, None].expand(-1, H, -1)
    k = _padded(torch.cat((st["k"].float(), shared), -1), ks, st["max_key_len"]).transpose(1, 2)
    v = _padded(st["v"].float(), ks, st["max_key_len"]).transpose(1, 2)
    i = torch.arange(st["max_query_len"], device="cuda")
    t = torch.arange(st["max_key_len"], device="cuda")
    z = torch.matmul(q, k.transpose(-1, -2)) * st["scale"]
    seen = (t <= (nk - nq)[:, None, None] + i[:, None]) & (t < nk[:, None, None])
    z = z.masked_fill(~seen[:, None], -math.inf)
    e = torch.exp(z - z.amax(-1, keepdim=True))
    o = torch.matmul(e, v) / e.sum(-1, keepdim=True)
    st["out"].copy_(_ragged(o.transpose(1, 2), qs, st["q"].shape[0]))
    return st["out"]


def _plain_decode(st):
    c = st["case"]
    S, H, R = c["S"], c["H"], c["R"]
    starts, ctx = st["query_start"].long(), st["context_lens"].long()
    n = st["max_query_len"]
    new = starts[1:] - starts[:-1]
    rows = st["cache"][st["tables"].long().clamp(min=0)].flatten(1, 2).float()  # [S, tokens, R+P]
    q = _padded(st["q"], starts, n).float().flatten(1, 2)                       # [S, new H, R+P]
    z = torch.matmul(q, rows.transpose(-1, -2)).view(S, n, H, -1) * st["scale"]
    t = torch.arange(rows.shape[1], device="cuda")
    at = t - (ctx - new)[:, None]                         # place among the new tokens, or negative
    if st["ancestors"] is None:
        seen = at[:, None] <= torch.arange(n, device="cuda")[:, None]
    else:
        bits = _padded(st["ancestors"], starts, n)[..., None]
        seen = (at[:, None] < 0) | ((bits >> at[:, None].clamp(0, 63)) & 1 == 1)
    seen = seen & (t < ctx[:, None, None])
    z = z.masked_fill(~seen[:, :, None], -math.inf)
    e = torch.exp(z - z.amax(-1, keepdim=True))
    o = torch.matmul(e.flatten(1, 2), rows[..., :R]).view(S, n, H, R) / e.sum(-1, keepdim=True)
    st["out"].copy_(_ragged(o, starts, st["q"].shape[0]))
    return st["out"]


# ------------------------------------------------------------------- 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    return {"write": _exact_write, "gather": _exact_gather, "prompt": _exact_prompt,
            "decode": _exact_decode}[case["op"]](st)


def _exact_write(st):
    c = st["case"]
    # each pair as a complex number, multiplied by the unit number of its angle
    unit = torch.polar(torch.full_like(st["inv_freq"], st["rope_scale"])[None],
                       st["positions"].double()[:, None] * st["inv_freq"][None])
    first = torch.arange(0, P, 2) if c["interleaved"] else torch.arange(P // 2)
    second = first + (1 if c["interleaved"] else P // 2)

    def turned(x, unit):
        y = x.double()
        z = torch.complex(y[..., first], y[..., second]) * unit
        y[..., first], y[..., second] = z.real, z.imag
        return y

    x = st["latent"].double()
    if st["weight"] is not None:
        x = x * (x.pow(2).sum(-1, keepdim=True) / c["R"] + st["eps"]).rsqrt() * st["weight"].double()
    cache = st["cache"].double()
    flat = cache.view(-1, c["R"] + P)
    flat[st["slots"], :c["R"]] = x
    flat[st["slots"], c["R"]:] = turned(st["k_rope"], unit)
    return turned(st["q"], unit[:, None]), cache


def _exact_gather(st):
    B, starts = st["case"]["B"], st["key_start"].tolist()
    parts = []
    for s in range(len(starts) - 1):
        n = starts[s + 1] - starts[s]
        blocks = st["tables"][s, :-(-n // B)].long()
        parts.append(st["cache"].index_select(0, blocks).flatten(0, 1)[:n].double())
    return torch.cat(parts)


def _exact_prompt(st):
    N = st["case"]["N"]
    qs, ks = st["query_start"].tolist(), st["key_start"].tolist()
    out = torch.empty(st["out"].shape, dtype=torch.float64, device="cuda")
    for s in range(len(qs) - 1):
        rows, keys = slice(qs[s], qs[s + 1]), slice(ks[s], ks[s + 1])
        i = torch.arange(qs[s + 1] - qs[s], device="cuda")[:, None]
        t = torch.arange(ks[s + 1] - ks[s], device="cuda")[None]
        hidden = t - i > len(t[0]) - len(i)
        for h in range(st["case"]["H"]):
            q = st["q"][rows, h].double()
            z = q[:, :N] @ st["k"][keys, h].double().T + q[:, N:] @ st["k_rope"][keys].double().T
            z = (z * st["scale"]).masked_fill(hidden, -math.inf)
            out[rows, h] = torch.softmax(z, -1) @ st["v"][keys, h].double()
    return out


def _exact_decode(st):
    c = st["case"]
    starts, ctx = st["query_start"].tolist(), st["context_lens"].tolist()
    out = torch.empty(st["out"].shape, dtype=torch.float64, device="cuda")
    for s, n in enumerate(ctx):
        token = torch.arange(n, device="cuda")
        rows = st["cache"][st["tables"][s].long()[token // c["B"]], token % c["B"]].double()
        m = starts[s + 1] - starts[s]
        for i in range(m):
            drafted = token - (n - m)
            if st["ancestors"] is None:
                seen = drafted <= i
            else:
                bits = int(st["ancestors"][starts[s] + i])
                path = [j for j in range(m) if bits >> j & 1]
                seen = (drafted < 0) | torch.isin(drafted, torch.tensor(path, device="cuda"))
            mine = rows[seen]
            z = st["q"][starts[s] + i].double() @ mine.T * st["scale"]
            out[starts[s] + i] = torch.softmax(z, -1) @ mine[:, :c["R"]]
    return out
