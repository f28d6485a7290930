"""Outputs that the calls of the 4-bit cache refuse: half a pair, memory of the cache itself."""
import pytest

pytestmark = pytest.mark.gpu


def _ints(v):
    import torch
    return torch.tensor(list(v), dtype=torch.int32, device="cuda")


def test_load_takes_both_outputs_or_none(cuda):
    import torch
    from depth_recurrent_attention_b200.attention import KV4Cache
    c = KV4Cache.alloc(1, 2, 64, 64)
    x = torch.randn((6, 2, 64), device="cuda").bfloat16()
    cu, start = _ints([0, 6]), _ints([0])
    c.store(x, x, cu, start)
    o = torch.full_like(x, 5.0)
    for pair in ((o, None), (None, o)):
        with pytest.raises(ValueError):
            c.load(cu, start, 6, out=pair)
    assert (o == 5).all()
    k, v = c.load(cu, start, 6, out=(None, None))
    assert torch.equal(k, v) and (k != 0).any()


def test_memory_of_the_cache_is_no_output(cuda):
    """Nor what is stored: rows inside the cache's tensor, at its ends, of another depth."""
    import torch
    from depth_recurrent_attention_b200.attention import KV4Cache
    buf = torch.zeros(16384 + 2 * 4 * 4608 + 16384, dtype=torch.uint8, device="cuda")
    c = KV4Cache(buf[16384:-16384].view(2, 2, 2, 1, 4608), 64)
    cu, start, lens = _ints([0, 1, 2]), _ints([0, 0]), _ints([1, 1])
    ok = torch.ones((2, 2, 64), device="cuda").bfloat16()

    def at(byte):
        return buf[byte:byte + 512].view(torch.bfloat16).view(2, 2, 64)

    size = 2 * 4 * 4608
    for byte in (16384 - 496, 16384, 16384 + size // 2, 16384 + size - 16):
        x = at(byte)
        for fn, args, kw in ((c.store, (x, ok, cu, start), {}), (c.store, (ok, x, cu, start), {}),
                             (c.load, (cu, start, 2), dict(out=(x, ok))), (c.load, (cu, start, 2), dict(out=(ok, x))),
                             (c.attend, (ok, lens), dict(out=x))):
            with pytest.raises(ValueError):
                fn(*args, **kw)
    assert not buf.any()
    for byte in (16384 - 512, 16384 + size):                    # right before it and behind it
        x = at(byte)
        x.copy_(torch.randn((2, 2, 64), device="cuda"))
        c.store(x, x, cu, start)
        k, _ = c.load(cu, start, 2, out=(x, ok))
        assert k is x and c.attend(ok, lens, out=x) is x
        # one key: its value is the output
        want = c.load(cu, start, 2)[1]
        assert torch.equal(x, want)


def test_boundaries_and_starts_at_the_ends_of_32_bits(cuda):
    """A first boundary far below 0 (rows behind it belong to the sequence) and a start near 2^31: the position
    is their sum, outside the cache, and nothing wraps around into it."""
    import torch
    from depth_recurrent_attention_b200.attention import KV4Cache
    c = KV4Cache.alloc(1, 2, 64, 64)
    x = torch.randn((4, 2, 64), device="cuda").bfloat16()
    for first, start in ((-2 ** 31, 2 ** 31 - 1), (-2 ** 31, 2 ** 31 - 4), (-2 ** 31, -5), (-9, 2 ** 31 - 1)):
        st = _ints([0])
        c.store(x, x, _ints([first, 4]), _ints([start]), status=st)
        assert st.item() != 0 and not c.data.any(), (first, start)
    st = _ints([0])
    c.store(x, x, _ints([-9, 4]), _ints([3]), status=st)       # row 0 is the sequence's tenth
    k, _ = c.load(_ints([0, 4]), _ints([12]), 4)
    assert st.item() == 0 and (k != 0).any(-1).all()
