"""Scores of any finite size: one far above the others (or several equally far) takes the row,
whatever its sign and size, as in the definition.

The score lies in 16 equal elements of the rotated part, q0 * key each, beside zeros, so it is
exact in fp32 before the scale, and the ones behind the largest are smaller by a tenth of the
largest and more: far past any rounding.  The weights that remain are the largest one's, 2^k, and
equal ones': sums, quotients and the join's factors are exact, and so is the expected row, the
value (or the mean of two, rounded once)."""
import numpy as np
import pytest

from helpers import to_dev
import oracle.latent as L
from latent_helpers import P, check, decode_case, on_device, prefill_case, run_decode
from paged_kv_cache_05_gb300 import workloads as W

pytestmark = pytest.mark.gpu

# of the largest score, natural; 16 products of fp16 elements reach 1.6e10 before the scale
SIZES = {"f16": [3e3, 1e5, 4e6, 4.5e7, 6e7, 9.4e7, 1.3e8, 1.9e8, 3.7e8, 5.4e8, 1e9],
         "bf16": [1e5, 6e7, 5e8, 4e9, 1e13, 1e20, 1e30]}


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_05_gb300 import build
    build.build()
    import paged_kv_cache_05_gb300 as m
    return m


def keys_of(rs, n, kind, sign, dtype):
    """n keys and the indexes of the largest scores (q0 > 0), as (float32 [n], list)."""
    import torch
    if kind == "ascending":                     # the maximum rises in every step
        far = np.linspace(0.05, 0.9, n)
        at = [n - 1]
    else:
        far = rs.uniform(0.1, 0.9, n)
        at = [int(rs.randint(n))] if kind == "one" else sorted(rs.choice(n, min(n, 2), False).tolist())
    k = far if sign > 0 else -(2 - far)
    k[at] = sign
    t = torch.from_numpy(k.astype(np.float32)).to(W.torch_dtype(dtype))
    return t, at


def factors(size, dtype, scale):
    """q0 and what the keys are multiplied by: `size` / |scale| in 16 products."""
    both = size / abs(scale) / 16
    q0 = 2.0 ** np.floor(np.log2(both) / 2)
    k = 2.0 ** np.floor(np.log2(both / q0))
    if dtype == "f16":
        q0 = min(q0, 32768.0)
        k = min(2.0 ** np.floor(np.log2(both / q0)), 16384.0)
    return q0, k * min(max(both / q0 / k, 1.0), 1.9)


def cases(dtype):
    return [(size, kind, sign) for size in SIZES[dtype] for kind in ("one", "two", "ascending")
            for sign in (1, -1)]


def expect(v, at, dtype):
    import torch
    return v[at].float().mean(0).to(W.torch_dtype(dtype)) if len(at) > 1 else v[at[0]]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("H,R,ctx", [(4, 512, 100), (3, 256, 1), (16, 512, 3000), (200, 256, 1500),
                                     (5, 256, 2000)])
@pytest.mark.parametrize("scale", [0.07, -0.11])
def test_absorbed(pkv, dtype, H, R, ctx, scale):
    import torch
    rs = np.random.RandomState(H + ctx)
    c = decode_case(rs, H, R, 16, [1], [ctx], dtype)
    d = on_device(c)
    blocks = d["bt"][0, :-(-ctx // 16)].long()
    rows = d["cache"][blocks].view(-1, R + P)[:ctx].clone()
    for size, kind, sign in cases(dtype):
        k, at = keys_of(rs, ctx, kind, sign, dtype)
        q0, by = factors(size, dtype, scale)
        rows[:, R:] = 0
        rows[:, R + 7:R + 23] = (k.float() * by).to(rows.dtype).cuda()[:, None]
        full = d["cache"][blocks].view(-1, R + P)
        full[:ctx] = rows
        d["cache"][blocks] = full.view(-1, 16, R + P)
        d["q"].zero_()
        d["q"][..., R + 7:R + 23] = q0 if scale > 0 else -q0
        got = run_decode(pkv, c, scale, d)
        assert pkv.get_device_error() == 0
        want = expect(rows[:, :R], at, dtype)
        assert torch.equal(got[0], want.expand(H, R)), (size, kind, sign)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("H,N,new,keys", [(2, 128, 3, 60), (1, 64, 1, 1), (2, 64, 300, 500), (4, 128, 2, 3000),
                                          (2, 64, 520, 2000)])
@pytest.mark.parametrize("scale", [0.07, -0.11])
def test_expanded(pkv, dtype, H, N, new, keys, scale):
    import torch
    rs = np.random.RandomState(N + keys)
    c = prefill_case(rs, H, N, [new], [keys], dtype)
    q, up, r = (to_dev(c[n], dtype) for n in ("q", "up", "rows"))
    q, up, r = q[:new], up[:keys], r[:keys, c["pad"]:].contiguous()
    starts = [torch.tensor([0, n], dtype=torch.int32, device="cuda") for n in (new, keys)]
    first = keys - new + 1                       # keys that every row sees
    for size, kind, sign in cases(dtype):
        if kind == "ascending":
            k, at = keys_of(rs, keys, kind, sign, dtype)
        else:                                    # the largest among those that every row sees
            k, at = keys_of(rs, first, kind, sign, dtype)
            more = rs.uniform(0.1, 0.8, keys - first).astype(np.float32)
            more = torch.from_numpy(more if sign > 0 else more - 2).to(k.dtype)
            k = torch.cat([k, more])
        q0, by = factors(size, dtype, scale)
        r.zero_()
        r[:, 7:23] = (k.float() * by).to(r.dtype).cuda()[:, None]
        q.zero_()
        q[..., N + 7:N + 23] = q0 if scale > 0 else -q0
        out = torch.full((new, H, N), 7.0, dtype=q.dtype, device="cuda")
        pkv.latent_attention_prefill(out, q, up[..., :N], r, up[..., N:], *starts, scale, new, keys)
        assert pkv.get_device_error() == 0
        if kind == "ascending":
            last = r[:, 7].float()
            # (neighbours differ by 2^-11 of the score, too little at the smallest)
            for i in {0, new // 2, new - 1} if size > 5e4 else {new - 1}:
                t = keys - new + i
                mine = (last[:t + 1] == last[:t + 1].max()).nonzero()[:, 0].tolist()
                if len(mine) < 3:
                    assert torch.equal(out[i], expect(up[..., N:], mine, dtype)), (size, kind, sign, i)
        else:
            want = expect(up[..., N:], at, dtype)
            assert torch.equal(out, want.expand(new, H, N)), (size, kind, sign)


def offset_scores(rs, n, dtype, size, scale):
    """Two elements of n keys and of the query: a part of `size` that all share, and scores of
    a few units on it."""
    import torch
    q0, k0 = factors(size * 16, dtype, scale)
    t = W.torch_dtype(dtype)
    keys = torch.empty((n, 2)).to(t)
    keys[:, 0] = k0
    keys[:, 1] = torch.from_numpy(rs.randn(n).astype(np.float32) * 3 / abs(scale)).to(t)
    return torch.tensor([q0 if scale > 0 else -q0, 1.0]).to(t), keys


# The scores are two products; adding them in fp32 and scaling the sum is off by a half step of
# it each, 2^-24 of the score, and so are its difference from the maximum, the maximum itself and
# the factors between maxima of different steps and parts, in log2 units: less than 2^-20 of the
# score in all.
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("size", [3e3, -3e3, 6e4, -3e5])
@pytest.mark.parametrize("scale", [0.07, -0.11])
def test_far_from_zero(pkv, dtype, size, scale):
    import torch
    rs = np.random.RandomState(int(abs(size)))
    dz = 2.0 ** -20 * abs(size) + 48 * 2.0 ** -20
    f = lambda x: x.double().cpu().numpy()                                      # noqa: E731
    for H, R, ctx in ((4, 512, 2000), (200, 256, 300)):
        c = decode_case(rs, H, R, 16, [1], [ctx], dtype)
        d = on_device(c)
        qe, keys = offset_scores(rs, ctx, dtype, abs(size), scale)
        blocks = d["bt"][0, :-(-ctx // 16)].long()
        full = d["cache"][blocks].view(-1, R + P)
        full[:ctx, R:] = 0
        full[:ctx, [R + 7, R + 40]] = keys.cuda() * torch.tensor([1 if size > 0 else -1, 1], device="cuda")
        d["cache"][blocks] = full.view(-1, 16, R + P)
        d["q"].zero_()
        d["q"][..., [R + 7, R + 40]] = qe.cuda()
        got = run_decode(pkv, c, scale, d)
        assert pkv.get_device_error() == 0
        q, rows = f(d["q"]), f(full[:ctx])
        ref, big = (L.prefill(q, np.repeat(k[:, None, :R], H, 1) * 0, rows[:, R:],
                              np.repeat(k[:, None, :R], H, 1), [0, 1], [0, ctx], scale)
                    for k in (rows, np.abs(rows)))
        check(got, ref, dtype, dz, big, ctx)
    for H, N, new, keys_n in ((2, 128, 60, 400), (2, 64, 3, 2000)):
        c = prefill_case(rs, H, N, [new], [keys_n], dtype)
        q, up, r = (to_dev(c[n], dtype) for n in ("q", "up", "rows"))
        q, up, r = q[:new], up[:keys_n], r[:keys_n, c["pad"]:].contiguous()
        qe, keys = offset_scores(rs, keys_n, dtype, abs(size), scale)
        r.zero_()
        r[:, [7, 40]] = keys.cuda() * torch.tensor([1 if size > 0 else -1, 1], device="cuda")
        q.zero_()
        q[..., [N + 7, N + 40]] = qe.cuda()
        starts = [torch.tensor([0, n], dtype=torch.int32, device="cuda") for n in (new, keys_n)]
        out = torch.full((new, H, N), 7.0, dtype=q.dtype, device="cuda")
        pkv.latent_attention_prefill(out, q, up[..., :N], r, up[..., N:], *starts, scale, new, keys_n)
        assert pkv.get_device_error() == 0
        k, v = f(up[..., :N]), f(up[..., N:])
        ref, big = (L.prefill(f(q), k, f(r), x, [0, new], [0, keys_n], scale) for x in (v, np.abs(v)))
        check(out, ref, dtype, dz, big, keys_n)
