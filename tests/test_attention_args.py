"""Argument checks of the handle-free attention operators, before any device call (no GPU)."""
import ctypes as C

import pytest


@pytest.fixture(scope="module")
def L():
    from depth_recurrent_attention_b200 import build
    build.build()
    from depth_recurrent_attention_b200 import attention
    return attention._lib()


def test_kv4_bytes(L):
    assert L.dreamer_kv4_bytes(2, 3, 64, 128) == 2 * 3 * 2 * 4608
    assert L.dreamer_kv4_bytes(1, 1, 128, 64) == 9216
    assert L.dreamer_kv4_bytes(64, 16, 128, 1 << 20) == 64 * 16 * (1 << 14) * 9216
    for bad in ((0, 1, 64, 64), (1, 0, 64, 64), (1, 1, 96, 64), (1, 1, 64, 65), (1, 1, 64, 0)):
        assert L.dreamer_kv4_bytes(*bad) == 0


P = 1 << 20   # a 16-byte aligned address that no refused call reads


def _cache(**kw):
    from depth_recurrent_attention_b200.attention import KV4CacheC
    f = dict(data=P, batch=2, n_kv_heads=2, head_dim=64, capacity=128)
    f.update(kw)
    return C.byref(KV4CacheC(*f.values()))


ARG, UNS = -1, -2


@pytest.mark.parametrize("kw,rc", [
    (dict(data=None), ARG), (dict(data=P + 8), ARG), (dict(batch=0), ARG), (dict(n_kv_heads=0), ARG),
    (dict(capacity=0), ARG), (dict(capacity=100), UNS), (dict(head_dim=32), UNS), (dict(head_dim=256), UNS),
    (dict(batch=1 << 20, n_kv_heads=64), UNS),
])
def test_caches_that_are_refused(L, kw, rc):
    c = _cache(**kw)
    assert L.dreamer_kv4_store(c, P, 1 << 12, P, 1 << 12, P, P, 4, 1, None, None) == rc
    assert L.dreamer_kv4_load(c, P, 1 << 12, P, 1 << 12, P, P, 4, 1, 0, None, None) == rc
    assert L.dreamer_attn_kv4(c, P, 1 << 12, P, 1 << 12, P, 4 if kw.get("n_kv_heads") != 64 else 64, 1, 0.125,
                              P, 1 << 40, None, None) == rc


@pytest.mark.parametrize("at,value", [
    (1, None), (1, P + 2), (2, 127), (2, 132), (3, None), (3, P + 4), (4, 64), (5, None), (6, None),
    (7, -1), (8, 2), (8, -1),
])
def test_rows_that_are_refused(L, at, value):
    a = [_cache(), P, 128, P, 128, P, P, 4, 1, None, None]
    a[at] = value
    assert L.dreamer_kv4_store(*a) == ARG
    assert L.dreamer_kv4_load(*a[:9], 0, *a[9:]) == ARG


@pytest.mark.parametrize("at,value", [
    (1, None), (1, P + 2), (2, 127), (2, 260), (3, None), (3, P + 4), (4, 64), (5, None), (6, 3), (6, 0),
    (7, 2), (8, float("nan")), (8, float("inf")),
])
def test_attention_calls_that_are_refused(L, at, value):
    a = [_cache(), P, 256, P, 256, P, 4, 1, 0.125, None, 0, None, None]
    a[at] = value
    assert L.dreamer_attn_kv4(*a) == ARG
    assert L.dreamer_attn_kv4(None, *a[1:]) == ARG


def test_no_rows_is_no_work(L):
    assert L.dreamer_kv4_store(_cache(), P, 128, P, 128, P, P, 0, 1, None, None) == 0
    assert L.dreamer_kv4_load(_cache(), P, 128, P, 128, P, P, 0, 1, 0, None, None) == 0


def test_the_binding_refuses_tensors_of_the_host():
    import torch
    from depth_recurrent_attention_b200.attention import KV4Cache
    with pytest.raises(ValueError):
        KV4Cache(torch.zeros((1, 1, 1, 1, 4608), dtype=torch.uint8), 64)
    with pytest.raises(ValueError):
        KV4Cache.alloc(1, 1, 96, 64)
    with pytest.raises(ValueError):
        KV4Cache.alloc(0, 1, 64, 64)


# q ldq k ldk v ldv out ldo cu n_seq n_tokens Hq Hkv d dtype scale status stream
PACKED = [P, 256, P, 128, P, 128, P, 256, P, 2, 10, 4, 2, 64, 1, 0.125, None, None]


@pytest.mark.parametrize("at,value,rc", [
    (0, None, ARG), (2, None, ARG), (4, None, ARG), (6, None, ARG), (8, None, ARG), (0, P + 8, ARG),
    (1, 255, ARG), (1, 260, ARG), (3, 127, ARG), (5, 64, ARG), (7, 128, ARG), (1, 1 << 40, ARG),
    (9, -1, ARG), (10, -1, ARG), (11, 3, ARG), (11, 0, ARG), (12, 0, ARG), (13, 0, ARG), (14, 2, ARG),
    (15, 0.0, ARG), (15, -1.0, ARG), (15, float("nan"), ARG), (15, float("inf"), ARG),
    (13, 32, UNS), (13, 96, UNS), (13, 256, UNS),
])
def test_packed_calls_that_are_refused(L, at, value, rc):
    a = list(PACKED)
    a[at] = value
    assert L.dreamer_attn_packed(*a) == rc


def test_packed_without_rows_or_prompts_is_no_work(L):
    for at in (9, 10):
        a = list(PACKED)
        a[at] = 0
        assert L.dreamer_attn_packed(*a) == 0


def test_the_packed_binding_refuses_tensors_of_the_host():
    import torch
    from depth_recurrent_attention_b200.attention import attn_packed
    x = torch.zeros((4, 1, 64))
    with pytest.raises(ValueError):
        attn_packed(x, x, x, torch.zeros(2, dtype=torch.int32))


def test_workspace_of_attention(L):
    small, large = _cache(), _cache(batch=2, n_kv_heads=2, capacity=1 << 15)
    assert L.dreamer_attn_kv4_workspace(small, 4) == 0
    need = L.dreamer_attn_kv4_workspace(large, 16)
    assert need > 0 and L.dreamer_attn_kv4_workspace(large, 17) == 0 and L.dreamer_attn_kv4_workspace(None, 16) == 0
    a = [large, P, 1 << 12, P, 1 << 12, P, 16, 1, 0.125, None, 0, None, None]
    for ws, n in ((None, need), (P, need - 1), (P + 8, need)):
        a[9], a[10] = ws, n
        assert L.dreamer_attn_kv4(*a) == ARG
