"""What the Python entry points of the attention operators refuse, and the memory they return."""
import sys

import pytest

pytestmark = pytest.mark.gpu


def _ints(v):
    import torch
    return torch.tensor(list(v), dtype=torch.int32, device="cuda")


def _args(**kw):
    import torch
    z = dict(dtype=torch.bfloat16, device="cuda")
    a = dict(q=torch.ones((6, 4, 64), **z), k=torch.ones((6, 2, 64), **z), v=torch.ones((6, 2, 64), **z),
             cu_seqlens=_ints([0, 2, 6]))
    a.update(kw)
    return a


BAD_PACKED = {
    "q of the host": lambda t: dict(q=t.ones((6, 4, 64))),
    "no tensor": lambda t: dict(k=None),
    "a list": lambda t: dict(cu_seqlens=[0, 2, 6]),
    "two dimensions": lambda t: dict(q=t.ones((6, 256), dtype=t.bfloat16, device="cuda")),
    "float16": lambda t: dict(q=t.ones((6, 4, 64), dtype=t.float16, device="cuda")),
    "types that differ": lambda t: dict(k=t.ones((6, 2, 64), device="cuda")),
    "rows that differ": lambda t: dict(v=t.ones((5, 2, 64), dtype=t.bfloat16, device="cuda")),
    "heads that differ": lambda t: dict(v=t.ones((6, 1, 64), dtype=t.bfloat16, device="cuda")),
    "dims that differ": lambda t: dict(k=t.ones((6, 2, 32), dtype=t.bfloat16, device="cuda")),
    "heads without a group": lambda t: dict(q=t.ones((6, 3, 64), dtype=t.bfloat16, device="cuda")),
    "no heads": lambda t: dict(q=t.ones((6, 0, 64), dtype=t.bfloat16, device="cuda")),
    "heads apart": lambda t: dict(q=t.ones((6, 4, 128), dtype=t.bfloat16, device="cuda")[..., :64]),
    "heads first": lambda t: dict(q=t.ones((4, 6, 64), dtype=t.bfloat16, device="cuda").transpose(0, 1)),
    "repeated rows": lambda t: dict(q=t.ones((1, 4, 64), dtype=t.bfloat16, device="cuda").expand(6, 4, 64)),
    "rows off 16 bytes": lambda t: dict(q=t.ones((6, 4 * 64 + 4), dtype=t.bfloat16, device="cuda")[:, :256].view(6, 4, 64)),
    "a start off 16 bytes": lambda t: dict(q=t.ones(6 * 256 + 4, dtype=t.bfloat16, device="cuda")[4:].view(6, 4, 64)),
    "boundaries of 64 bits": lambda t: dict(cu_seqlens=t.tensor([0, 2, 6], device="cuda")),
    "boundaries of the host": lambda t: dict(cu_seqlens=t.tensor([0, 2, 6], dtype=t.int32)),
    "boundaries apart": lambda t: dict(cu_seqlens=_ints([0, 0, 2, 0, 6, 0])[::2]),
    "no boundaries": lambda t: dict(cu_seqlens=_ints([])),
    "an out of another shape": lambda t: dict(out=t.ones((6, 2, 64), dtype=t.bfloat16, device="cuda")),
    "an out of another type": lambda t: dict(out=t.ones((6, 4, 64), device="cuda")),
    "a scale of zero": lambda t: dict(scale=0.0),
    "a scale of nan": lambda t: dict(scale=float("nan")),
    "a scale past float32": lambda t: dict(scale=1e39),
    "a status of 64 bits": lambda t: dict(status=t.zeros(1, dtype=t.int64, device="cuda")),
    "a status of the host": lambda t: dict(status=t.zeros(1, dtype=t.int32)),
}


@pytest.mark.parametrize("what", BAD_PACKED)
def test_attn_packed_refuses(cuda, what):
    import torch
    from depth_recurrent_attention_b200.attention import attn_packed
    with pytest.raises(ValueError):
        attn_packed(**_args(**BAD_PACKED[what](torch)))


def test_out_beside_its_inputs_but_not_over_them(cuda):
    import torch
    from depth_recurrent_attention_b200.attention import attn_packed
    buf = torch.randn((50, 4 + 2 + 2 + 4, 64), device="cuda").bfloat16()
    q, k, v, out, cu = buf[:, :4], buf[:, 4:6], buf[:, 6:8], buf[:, 8:], _ints([0, 20, 50])
    want = attn_packed(q.clone(), k.clone(), v.clone(), cu)
    assert torch.equal(attn_packed(q, k, v, cu, out=out), want) and torch.equal(out, want)
    for bad in (q, buf[:, 1:5], buf[:, 4:8], buf[:, 5:9], buf[:, 7:11]):
        with pytest.raises(ValueError):
            attn_packed(q, k, v, cu, out=bad)
    rows = torch.randn((99, 4, 64), device="cuda").bfloat16()       # rows of one buffer
    one = _ints([0, 33])
    attn_packed(rows[:33], rows[33:66], rows[33:66], one, out=rows[66:])
    for first in (0, 1, 33, 65):
        with pytest.raises(ValueError):
            attn_packed(rows[:33], rows[33:66], rows[33:66], one, out=rows[first:first + 33])
    flat = torch.randn(40 * 320, device="cuda").bfloat16()          # strides that differ
    with pytest.raises(ValueError):
        attn_packed(q[:20], k[:20], v[:20], _ints([0, 20]), out=buf.view(-1)[:20 * 256].view(20, 4, 64))
    assert attn_packed(q[:20], k[:20], v[:20], _ints([0, 20]), out=flat[:20 * 256].view(20, 4, 64)).shape == (20, 4, 64)


def test_other_types_and_unsupported_dims(cuda):
    import torch
    from depth_recurrent_attention_b200.attention import attn_packed
    from depth_recurrent_attention_b200.dreamer import ERR_UNSUPPORTED, DreamerError
    with pytest.raises(TypeError):
        attn_packed(**_args(scale="1"))
    with pytest.raises(AttributeError):
        attn_packed(**_args(stream=5))
    x = torch.ones((6, 2, 32), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(DreamerError) as e:
        attn_packed(x, x, x, _ints([0, 6]))
    assert e.value.code == ERR_UNSUPPORTED


def test_the_cache_refuses(cuda):
    import torch
    from depth_recurrent_attention_b200.attention import KV4Cache
    c = KV4Cache.alloc(2, 2, 64, 128, depth=3)
    assert (c.depth, c.batch, c.n_kv_heads, c.capacity) == (3, 2, 2, 128)
    z = dict(dtype=torch.bfloat16, device="cuda")
    k, q, cu, start, lens = torch.ones((5, 2, 64), **z), torch.ones((2, 4, 64), **z), _ints([0, 2, 5]), _ints([0, 0]), _ints([2, 3])

    def refused(fn, *a, error=ValueError, **kw):
        with pytest.raises(error):
            fn(*a, **kw)

    refused(KV4Cache, c.data, 128)
    refused(KV4Cache, c.data, 32)
    refused(KV4Cache, c.data[..., :-1], 64)
    refused(KV4Cache, c.data[0], 64)
    refused(KV4Cache, c.data.view(torch.int8), 64)
    refused(KV4Cache, c.data.transpose(1, 2), 64)
    refused(KV4Cache, c.data[:0], 64)
    refused(KV4Cache, None, 64)
    for depth in (-1, 3):
        refused(c.store, k, k, cu, start, depth=depth)
        refused(c.load, cu, start, 5, depth=depth)
        refused(c.attend, q, lens, depth=depth)
    refused(c.store, k, k.float(), cu, start)
    refused(c.store, k, k[:4], cu, start)
    refused(c.store, k[:, :1], k[:, :1], cu, start)
    refused(c.store, k, k, cu[:2], start)
    refused(c.store, k, k, cu, cu)
    refused(c.store, k, k, cu.long(), start)
    refused(c.load, cu, start, -1)
    refused(c.load, cu, start, 5, dtype=torch.float16)
    refused(c.load, cu, start, 5, out=(k, k[:4]))
    refused(c.load, cu, start, 5, dtype=torch.float32, out=(k, k))
    refused(c.load, cu, start, 1.5, error=TypeError)
    refused(c.attend, q[:1], lens)
    refused(c.attend, q[:, :3].contiguous(), lens)
    refused(c.attend, q, cu)
    refused(c.attend, q, lens, out=q[:, :2])
    refused(c.attend, q, lens, scale=float("inf"))
    wide = torch.ones((2, 6, 64), **z)
    refused(c.attend, wide[:, :4], lens, out=wide[:, 2:])
    refused(c.load, cu, start, 5, out=(k, k))
    refused(c.attend, q, lens, status=torch.zeros(1, device="cuda"))
    assert not c.data.any()                      # nothing was written


def test_attend_in_place(cuda):
    import torch
    from depth_recurrent_attention_b200.attention import KV4Cache
    for cap in (64, 64 * 200):                  # one launch, and a split with a join
        c = KV4Cache.alloc(2, 2, 64, cap)
        k = torch.randn((100, 2, 64), device="cuda").bfloat16()
        c.store(k, k.flip(0), _ints([0, 60, 100]), _ints([0, 0]))
        q = torch.randn((2, 4, 64), device="cuda").bfloat16()
        want = c.attend(q, _ints([60, 40]))
        assert c.attend(q, _ints([60, 40]), out=q) is q and torch.equal(q, want)


def test_no_rows(cuda):
    import torch
    from depth_recurrent_attention_b200.attention import KV4Cache, attn_packed
    e = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    assert attn_packed(e, e, e, _ints([0])).shape == (0, 2, 64)
    assert attn_packed(e, e, e, _ints([0, 0])).shape == (0, 2, 64)
    c = KV4Cache.alloc(1, 2, 64, 64)
    c.store(e, e, _ints([0, 0]), _ints([0]))
    k, v = c.load(_ints([0, 0]), _ints([0]), 0)
    assert k.shape == v.shape == (0, 2, 64) and not c.data.any()


def test_one_row_of_any_stride(cuda):
    import torch
    from depth_recurrent_attention_b200.attention import attn_packed
    x = torch.randn((1, 2, 64), device="cuda").bfloat16()
    odd = torch.as_strided(x, (1, 2, 64), (7, 64, 1))
    assert torch.equal(attn_packed(odd, odd, odd, _ints([0, 1])), x)   # one key: its value


def test_out_is_returned_itself_and_references_are_kept_even(cuda):
    import torch
    from depth_recurrent_attention_b200.attention import KV4Cache, attn_packed
    a = _args(out=torch.zeros((6, 4, 64), dtype=torch.bfloat16, device="cuda"))
    c = KV4Cache.alloc(1, 2, 64, 64)
    one, zero = _ints([0, 6]), _ints([0])
    pair = (torch.empty_like(a["k"]), torch.empty_like(a["v"]))
    q, lens, o = a["q"][:1].clone(), _ints([6]), torch.empty_like(a["q"][:1])
    held = [*a.values(), one, zero, pair[0], pair[1], q, lens, o, c.data]
    refs = [sys.getrefcount(x) for x in held]
    for _ in range(10):
        assert attn_packed(**a) is a["out"]
        c.store(a["k"], a["v"], one, zero)
        k, v = c.load(one, zero, 6, out=pair)
        assert k is pair[0] and v is pair[1]
        assert c.attend(q, lens, out=o) is o
        with pytest.raises(ValueError):
            attn_packed(**dict(a, scale=-1.0))
    del k, v
    assert [sys.getrefcount(x) for x in held] == refs


def test_new_memory_belongs_to_the_stream_of_the_call(cuda):
    """Blocks that a call allocates on a side stream go back to that stream's pool: the same call
    again reuses them, and the default stream's allocations never do."""
    import torch
    from depth_recurrent_attention_b200.attention import attn_packed
    a, s = _args(), torch.cuda.Stream()
    torch.cuda.synchronize()
    out = attn_packed(**a, stream=s)
    assert torch.cuda.current_stream() == torch.cuda.default_stream()
    p = out.data_ptr()
    del out
    others = [torch.empty((6, 4, 64), dtype=torch.bfloat16, device="cuda") for _ in range(64)]
    assert p not in [t.data_ptr() for t in others]
    with torch.cuda.stream(s):
        again = [torch.empty((6, 4, 64), dtype=torch.bfloat16, device="cuda") for _ in range(64)]
    assert p in [t.data_ptr() for t in again]
    s.synchronize()


def test_calls_wait_for_what_runs_before_them(cuda):
    """Inputs that a kernel, a copy or a fill writes just before the call, and outputs that a kernel still
    reads, with no synchronisation between: the same bits as with one after every step."""
    import torch
    from depth_recurrent_attention_b200.attention import KV4Cache, attn_packed
    g = torch.Generator("cuda").manual_seed(5)
    z = dict(device="cuda", generator=g)
    rows = [torch.randn((700, 4, 64), **z).bfloat16() for _ in range(3)]
    host = torch.randn((3, 8, 64), generator=torch.Generator().manual_seed(6)).bfloat16().pin_memory()
    cu, start, lens, heavy = _ints([0, 400, 401, 700]), _ints([0] * 3), _ints([400, 1, 299]), torch.randn((2048, 2048), **z)

    def steps(sync):
        c, got = KV4Cache.alloc(3, 4, 64, 64 * 80), []
        x, q, o = torch.zeros_like(rows[0]), torch.zeros((3, 8, 64), dtype=torch.bfloat16, device="cuda"), None
        for i in range(30):
            h = heavy @ heavy                       # the stream is busy: what follows queues up
            x.copy_(rows[i % 3])
            x[i] += h[0, 0].bfloat16() * 0 + 1      # written by a kernel
            sync()
            c.store(x, x.flip(0), cu, start)
            sync()
            x.fill_(9)                              # after the store has read it
            k, v = c.load(cu, start, 700)
            sync()
            o = attn_packed(k, v, k, cu, out=o)
            got.append(o.float().sum((1, 2)) + k.float().sum((1, 2)))
            sync()
            q.copy_(host, non_blocking=True)        # by a copy engine
            sync()
            got.append(c.attend(q, lens))
            q.zero_()
            sync()
        torch.cuda.synchronize()
        return got

    for a, b in zip(steps(lambda: None), steps(torch.cuda.synchronize)):
        assert torch.equal(a, b)
