"""Softmax scales that the attention operators refuse before any device call (no GPU)."""
import ctypes as C

import pytest

P = 1 << 20   # a 16-byte aligned address that no refused call reads


@pytest.mark.parametrize("scale", [3.4e38, 2.4e38])
def test_a_scale_that_log2_e_takes_out_of_float32(scale):
    from depth_recurrent_attention_b200 import attention, build
    build.build()
    L = attention._lib()
    assert L.dreamer_attn_packed(P, 256, P, 128, P, 128, P, 256, P, 2, 10, 4, 2, 64, 1, scale, None, None) == -1
    c = C.byref(attention.KV4CacheC(P, 2, 2, 64, 128))
    for s in (scale, -scale):
        assert L.dreamer_attn_kv4(c, P, 256, P, 256, P, 4, 1, s, None, 0, None, None) == -1
