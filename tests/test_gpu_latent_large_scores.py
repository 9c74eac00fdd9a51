"""Scores of any finite size: one far above the others (or several equally far) takes the row,
whatever its sign and size, as in the definition.

The score lies in 16 equal elements of the rotated part, q0 * key each, beside zeros, so it is
exact in fp32 before the scale, and the ones behind the largest are smaller by a tenth of the
largest and more: far past any rounding.  The weights that remain are the largest one's, 2^k, and
equal ones': sums, quotients and the join's factors are exact, and so is the expected row, the
value (or the mean of two, rounded once)."""
import numpy as np
import pytest

from latent_helpers import P, decode_case, on_device, run_decode
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
