"""Argument checks of the grouped attention entry points, without a GPU."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_05_gb300 import build
    build.build()
    import paged_kv_cache_05_gb300 as m
    return m


def test_workspace_size(pkv):
    size = pkv.decode_grouped_workspace_size
    assert 0 < size(1, 8, 8, 64, 16, 1) <= size(64, 40, 8, 128, 16, 128)
    assert size(64, 64, 4, 128, 16, 128) > size(64, 32, 4, 128, 16, 128)     # 16 heads a row
    for bad in [(-1, 8, 8, 64, 16, 4), (20000, 8, 8, 64, 16, 4), (4, 9, 2, 64, 16, 4),
                (4, 2, 4, 64, 16, 4), (4, 0, 0, 64, 16, 4), (4, 8, 0, 64, 16, 4),
                (4, 8, 2, 96, 16, 4), (4, 8, 2, 64, 24, 4), (4, 8, 2, 64, 16, 0),
                (1, 8, 2, 64, 16, (1 << 26) + 1), (16384, 8, 8, 128, 16, 1 << 20),
                (4, 1 << 17, 1, 64, 16, 4)]:
        with pytest.raises(pkv.PagedKVError) as e:
            size(*bad)
        assert e.value.status == 1


def test_decode_rejects_bad_arguments_before_any_gpu_call(pkv):
    L = pkv.lib()
    ws = ctypes.c_size_t(0)
    assert L.pkv_decode_grouped_workspace_size(4, 8, 2, 64, 16, 4, ctypes.byref(ws)) == 0
    f = 1 << 20                       # never dereferenced
    names = ["out", "q", "k", "v", "bt", "cl", "sl", "scale", "cap", "win", "S", "H", "HK", "D", "B",
             "maxb", "nb", "dtype", "ws", "wsb", "stream"]
    base = [f, f, f, f, f, f, None, 0.125, 0.0, 0, 4, 8, 2, 64, 16, 4, 64, 0, f * 256, ws.value,
            None]

    def call(**kw):
        a = list(base)
        for k, v in kw.items():
            a[names.index(k)] = v
        return L.pkv_paged_attention_decode_grouped(*a)

    for kw in [dict(D=80), dict(B=4), dict(nb=0), dict(nb=1 << 27), dict(dtype=3), dict(H=7),
               dict(HK=3), dict(HK=0), dict(S=-1), dict(maxb=0), dict(scale=float("inf")),
               dict(cap=-1.0), dict(cap=float("nan")), dict(cap=1e-42), dict(win=-1), dict(out=None),
               dict(bt=None), dict(cl=f + 2), dict(q=f + 8), dict(sl=f + 2), dict(ws=f * 256 + 128),
               dict(ws=None), dict(wsb=ws.value - 1)]:
        assert call(**kw) == 1, kw
        assert "grouped" in pkv.pagedkv.last_error()
    assert call(S=0) == 0


def test_prefill_rejects_bad_arguments_before_any_gpu_call(pkv):
    L = pkv.lib()
    f = 1 << 20
    names = ["out", "q", "k", "v", "bt", "cl", "qs", "sl", "scale", "cap", "win", "S", "H", "HK",
             "D", "B", "maxb", "nb", "most", "T", "dtype", "ws", "wsb", "stream"]
    base = [f, f, f, f, f, f, f, None, 0.125, 0.0, 0, 4, 8, 2, 64, 16, 4, 64, 10, 40, 0, None, 0,
            None]

    def call(**kw):
        a = list(base)
        for k, v in kw.items():
            a[names.index(k)] = v
        return L.pkv_paged_attention_prefill_grouped(*a)

    for kw in [dict(D=32), dict(B=128), dict(nb=0), dict(nb=1 << 27), dict(dtype=-1), dict(H=9),
               dict(HK=0), dict(S=-1), dict(S=70000), dict(maxb=0), dict(maxb=(1 << 26) + 1),
               dict(most=-1), dict(T=-1), dict(scale=float("nan")), dict(cap=-0.5), dict(win=-3),
               dict(out=None), dict(qs=None), dict(qs=f + 1), dict(v=f + 4), dict(sl=f + 1),
               dict(S=65535, H=65535, HK=65535, nb=1, maxb=1 << 26, most=(1 << 31) - 1)]:
        assert call(**kw) == 1, kw
        assert "grouped" in pkv.pagedkv.last_error()
    assert call(S=0) == 0 and call(T=0) == 0 and call(most=0) == 0
    # a workspace is looked at where the sizes may have use for it
    need = pkv.prefill_grouped_workspace_size(4, 8, 2, 64, 16, 64, 10)
    assert need > 0
    assert call(maxb=64, ws=f * 256, wsb=need - 1) == 1 and "small" in pkv.pagedkv.last_error()
    assert call(maxb=64, ws=f * 256 + 16, wsb=need) == 1
    for none in [(4, 8, 2, 64, 16, 4, 10), (4, 8, 2, 64, 16, 64, 100000), (4, 64, 2, 64, 16, 64, 500),
                 (1000, 8, 2, 64, 16, 64, 10)]:
        assert pkv.prefill_grouped_workspace_size(*none) == 0
    for bad in [(4, 7, 2, 64, 16, 64, 10), (4, 8, 2, 96, 16, 64, 10), (-1, 8, 2, 64, 16, 64, 10)]:
        with pytest.raises(pkv.PagedKVError):
            pkv.prefill_grouped_workspace_size(*bad)


def test_binding_refuses_host_tensors_and_other_objects(pkv):
    import torch
    t = torch.zeros(2, 2, 64, dtype=torch.float16)
    c = torch.zeros(1, 2, 16, 64, dtype=torch.float16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        pkv.norm_rope_and_cache(t, t, t, t, c, c, i.long(), i, None)
    with pytest.raises(ValueError):
        pkv.paged_attention_prefill_grouped(t, t, c, c, i.view(1, 2), i[:1], i, 0.1, 2)
    with pytest.raises(TypeError):
        pkv.norm_rope_and_cache(t, 3, t, t, c, c, i.long(), i, None)
    with pytest.raises(TypeError):
        pkv.paged_attention_prefill_grouped(t, t, c, c, i.view(1, 2), i[:1], i, "scale", 2)
