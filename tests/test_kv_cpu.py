"""The paged key/value cache's calls on the host: refusals before any launch, no-ops, workspace sizes (no GPU)."""
import ctypes

import pytest
import torch

from skinny_gemm_gb300 import ops

P = 0x10000  # a 256-byte aligned fake address, never dereferenced


@pytest.fixture()
def L(monkeypatch):
    monkeypatch.delenv("W4A16_FAULT", raising=False)
    lib = ops.lib()
    lib.w4a16_debug_reload_env()
    yield lib
    monkeypatch.delenv("W4A16_FAULT", raising=False)
    lib.w4a16_debug_reload_env()


def _cache(**over):
    f = dict(k=P, v=P, k_scale=P, v_scale=P, blocks=10, heads=2, block=16, dim=128)
    f.update(over)
    c = ops.KvCacheStruct(*(f[n] for n, _ in ops.KvCacheStruct._fields_))
    return ctypes.addressof(c), c


def _plan(L, head=None, **over):
    f = dict(cached=P, fresh=P, table=P, free=P, cu=P, lens=P, slots=P, pos=P, out=P + 4, B=3, T=5, block=16, max_blocks=4,
             n_free=9)
    f.update(over)
    return L.w4a16_kv_plan(f["cached"], f["fresh"], f["table"], f["free"], head, f["cu"], f["lens"], f["slots"], f["pos"],
                           f["out"], f["B"], f["T"], f["block"], f["max_blocks"], f["n_free"], None)


def test_plan_refusals(L, monkeypatch):
    for over in (dict(B=-1), dict(T=-1), dict(T=1 << 30), dict(block=0), dict(block=24), dict(block=256), dict(max_blocks=0),
                 dict(n_free=-1), dict(head=P + 4)):
        assert _plan(L, **over) == ops.ERR_SHAPE, over
    for name in ("cached", "fresh", "table", "free", "cu", "lens", "slots", "pos", "out"):
        assert _plan(L, **{name: None}) == ops.ERR_NULL, name
        assert _plan(L, **{name: P + 2}) == ops.ERR_ALIGN, name
    assert _plan(L, head=P + 1) == ops.ERR_ALIGN
    monkeypatch.setenv("W4A16_FAULT", "launch")
    L.w4a16_debug_reload_env()
    assert _plan(L) == ops.ERR_CUDA and _plan(L, block=17) == ops.ERR_SHAPE


def _append(L, cache=None, k=P, ks=256, v=P, vs=256, slots=P, T=3, **over):
    ptr, keep = _cache(**over)
    return L.w4a16_kv_append(k, ks, v, vs, slots, ptr if cache is None else cache, T, None)


BAD_CACHES = [dict(block=8), dict(block=48), dict(dim=96), dict(dim=512), dict(heads=0), dict(heads=70000), dict(blocks=0),
              dict(blocks=1 << 30, heads=2, block=16)]


def test_append_refusals(L, monkeypatch):
    assert _append(L, T=0, k=None, v=None, slots=None) == ops.OK
    for over in BAD_CACHES + [dict(T=-1), dict(T=1 << 30), dict(ks=248), dict(vs=128)]:
        assert _append(L, **over) == ops.ERR_SHAPE, over
    assert _append(L, cache=0) == ops.ERR_NULL
    for name in ("k", "v", "slots"):
        assert _append(L, **{name: None}) == ops.ERR_NULL, name
        assert _append(L, **{name: P + 2}) == ops.ERR_ALIGN, name
    assert _append(L, ks=260) == ops.ERR_ALIGN and _append(L, vs=257) == ops.ERR_ALIGN
    for name in ("k", "v"):  # the cache's own pointers
        ptr, keep = _cache(**{name: P + 8})
        assert L.w4a16_kv_append(P, 256, P, 256, P, ptr, 3, None) == ops.ERR_ALIGN
    for name in ("k", "v", "k_scale", "v_scale"):
        ptr, keep = _cache(**{name: None})
        assert L.w4a16_kv_append(P, 256, P, 256, P, ptr, 3, None) == ops.ERR_NULL
    monkeypatch.setenv("W4A16_FAULT", "validate")
    L.w4a16_debug_reload_env()
    assert _append(L) == ops.ERR_SHAPE


def _attend(L, cache_over=None, **over):
    f = dict(q=P, qs=1024, table=P, cu=P, lens=P, out=P, B=2, T=3, hq=8, max_blocks=4, max_new=2, max_len=64, window=0,
             scale=0.1, ws=P, wn=1 << 40)
    f.update(over)
    ptr, keep = _cache(**(cache_over or {}))
    return L.w4a16_kv_attention(f["q"], f["qs"], f.get("cache", ptr), f["table"], f["cu"], f["lens"], f["out"], f["B"],
                                f["T"], f["hq"], f["max_blocks"], f["max_new"], f["max_len"], f["window"], f["scale"],
                                f["ws"], f["wn"], f.get("counters", P), None)


def test_attention_refusals(L, monkeypatch):
    assert _attend(L, T=0, B=0, q=None, table=None, cu=None, lens=None, out=None, ws=None, wn=0) == ops.OK
    for over in BAD_CACHES:
        assert _attend(L, cache_over=over) == ops.ERR_SHAPE, over
    for over in (dict(B=-1), dict(T=-1), dict(B=0), dict(hq=7), dict(hq=0), dict(hq=66), dict(max_blocks=0), dict(max_new=0),
                 dict(max_len=0), dict(max_len=65), dict(window=-1), dict(scale=0.0), dict(scale=-1.0),
                 dict(scale=float("nan")), dict(scale=float("inf")), dict(qs=1016)):
        assert _attend(L, **over) == ops.ERR_SHAPE, over
    assert _attend(L, cache=None) == ops.ERR_NULL
    for name in ("q", "table", "cu", "lens", "out"):
        assert _attend(L, **{name: None}) == ops.ERR_NULL, name
        assert _attend(L, **{name: P + 2}) == ops.ERR_ALIGN, name
    assert _attend(L, qs=1028) == ops.ERR_ALIGN and _attend(L, out=P + 8) == ops.ERR_ALIGN
    assert _attend(L, ws=P + 128) == ops.ERR_ALIGN and _attend(L, counters=P + 2) == ops.ERR_ALIGN
    n = L.w4a16_kv_attention_workspace_bytes(2, 3, 8, 2, 128, 2, 64, 0)
    assert n > 0 and _attend(L, ws=None, wn=0) == ops.ERR_NULL and _attend(L, wn=n - 1) == ops.ERR_SHAPE
    assert _attend(L, counters=None) == ops.ERR_NULL
    monkeypatch.setenv("W4A16_FAULT", "launch")
    L.w4a16_debug_reload_env()
    assert _attend(L) == ops.ERR_CUDA and "injected" in L.w4a16_last_error().decode()


def test_workspace_query(L):
    f = L.w4a16_kv_attention_workspace_bytes
    assert f(0, 1, 8, 2, 128, 1, 64, 0) == 0 and f(1, 1, 7, 2, 128, 1, 64, 0) == 0 and f(1, 1, 8, 2, 96, 1, 64, 0) == 0
    a = f(4, 4, 8, 2, 128, 1, 5000, 0)
    assert a == f(4, 4, 8, 2, 128, 1, 5000, 0) and f(4, 4, 8, 2, 128, 1, 50000, 0) >= a
    assert f(4, 4, 8, 2, 128, 1, 50000, 512) <= f(4, 4, 8, 2, 128, 1, 50000, 0)


def test_workspace_query_refuses_what_the_call_refuses(L):
    """Too many query heads a key head; steps whose sizes pass 64 bits."""
    f = L.w4a16_kv_attention_workspace_bytes
    assert f(1, 1, 64, 2, 128, 1, 64, 0) > 0 and f(1, 1, 66, 2, 128, 1, 64, 0) == 0 and f(1, 1, 64, 1, 128, 1, 64, 0) == 0
    big = 2 ** 30 - 1
    assert f(big, big, 65535, 65535, 64, 1, 2 ** 31 - 1, 0) == 0 and f(big, big, 64, 2, 64, big, 2 ** 31 - 1, 0) == 0


def test_python_layer_checks_before_any_launch():
    bf, f8 = torch.bfloat16, torch.float8_e4m3fn
    with pytest.raises(ValueError):  # host tensors
        ops.KVCache(torch.zeros(2, 1, 16, 64, dtype=f8), torch.zeros(2, 1, 16, 64, dtype=f8), torch.zeros(2, 1), torch.zeros(2, 1))
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        ops.kv_plan(i, i, i, i, 4, 16)  # table is not [B, max_blocks]
    with pytest.raises(ValueError):
        ops.kv_plan(i, i, i.view(2, 1), i, 4, 16, out=ops.KVPlan.empty(2, 4, "cpu"))  # not on the GPU

    class Fake:
        heads, dim, block, _ptr = 2, 64, 16, 0

    x = torch.zeros(3, 2, 64, dtype=bf)
    with pytest.raises(ValueError):
        ops.kv_append(x, x, Fake(), i)
    with pytest.raises(ValueError):
        ops.kv_attention(x, Fake(), i.view(2, 1), i, i, 1, 16)
    with pytest.raises(ValueError):
        ops.kv_attention(x[0], Fake(), i.view(2, 1), i, i, 1, 16)
