"""Expired waits of the handle-free attention operators: the kernel reports, winds down and returns, what it
could not compute is marked, and the next call is right.

Runs the test-hook build of the library (20 ms wait limit): dreamer_test_withhold makes one warp of the
next call announce a copy into shared memory that it never makes, so that the wait for it runs out.
Nothing is in flight for that barrier when the blocks exit."""
import ctypes as C

import pytest

pytestmark = pytest.mark.gpu

TIMEOUT = 1


@pytest.fixture(scope="module")
def hooks(cuda):
    from depth_recurrent_attention_b200 import dreamer as D
    L = C.CDLL(D.TESTHOOKS_PATH)
    vp, i, i64, f = C.c_void_p, C.c_int, C.c_int64, C.c_float
    L.dreamer_attn_kv4.argtypes = [vp, vp, i64, vp, i64, vp, i, i, f, vp, i64, vp, vp]
    L.dreamer_attn_kv4_workspace.argtypes = [vp, i]
    L.dreamer_attn_kv4_workspace.restype = i64
    L.dreamer_attn_packed.argtypes = [vp, i64, vp, i64, vp, i64, vp, i64, vp, i, i, i, i, i, i, f, vp, vp]
    L.dreamer_test_withhold.argtypes = [i, i, i]
    return L


def _ints(v):
    import torch
    return torch.tensor(list(v), dtype=torch.int32, device="cuda")


def _attend(L, c, q, lens, out, status):
    import torch
    from depth_recurrent_attention_b200.attention import KV4CacheC
    cc = KV4CacheC(c.data.data_ptr(), c.batch, c.n_kv_heads, c.head_dim, c.capacity)
    need = L.dreamer_attn_kv4_workspace(C.byref(cc), q.shape[1])
    # what the workspace held before is no partial result of this call
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    w = q.shape[1] * q.shape[2]
    rc = L.dreamer_attn_kv4(C.byref(cc), q.data_ptr(), w, out.data_ptr(), w, lens.data_ptr(), q.shape[1],
                            0 if q.dtype == torch.float32 else 1, q.shape[2] ** -0.5,
                            ws.data_ptr() if need else None, need, status.data_ptr(), None)
    assert rc == 0
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("lens,H,capacity,at", [
    ([100, 200], 2, 256, (1, 0, 0)),                       # a CTA an item: the second head of the first sequence
    ([200, 200], 2, 256, (3, 3, 0)),
    ([300, 300], 2, 320, (3, 1, 0)),                       # two CTAs an item
    ([3000], 1, 3008, (2, 1, 0)),                          # a cluster of eight CTAs an item
    ([3000], 1, 3008, (7, 0, 0)),
    ([12800, 64, 12000, 700], 32, 12800, (0, 0, 1)),       # runs over all items: inside a long one,
    ([12800, 64, 12000, 700], 32, 12800, (100, 3, 0)),
    ([12800, 64, 12000, 700], 32, 12800, (270, 1, 0)),     # of short ones that a warp holds whole
    ([12800, 64, 12000, 700], 32, 12800, (540, 0, 0)),
])
def test_attend_after_an_expired_wait(hooks, dtype, lens, H, capacity, at):
    import torch
    from depth_recurrent_attention_b200.attention import KV4Cache
    torch.manual_seed(3)
    c = KV4Cache.alloc(len(lens), H, 64, capacity)
    n = sum(lens)
    k, v = torch.randn((2, n, H, 64), device="cuda")
    cu = [0]
    for x in lens:
        cu.append(cu[-1] + x)
    c.store(k, v, _ints(cu), _ints([0] * len(lens)))
    q = torch.randn((len(lens), H, 64), device="cuda").to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    ln, st = _ints(lens), _ints([0])
    good, out = torch.empty_like(q), torch.full_like(q, 5.0)
    _attend(hooks, c, q, ln, good, st)
    assert st.item() == 0 and torch.isfinite(good).all()
    cta, warp, copy = at
    if dtype == "fp32" and capacity > 10000:          # half as many warps, runs twice as long
        cta //= 2
    hooks.dreamer_test_withhold(cta, warp, copy)
    _attend(hooks, c, q, ln, out, st)
    assert st.item() == TIMEOUT
    lost = torch.isnan(out).all(-1)
    assert 1 <= int(lost.sum()) <= 32                 # what a CTA had in hand, no more
    assert torch.equal(out[~lost], good[~lost])
    st.zero_()
    _attend(hooks, c, q, ln, out, st)
    assert st.item() == 0 and torch.equal(out, good)


@pytest.mark.parametrize("d,at", [
    (64, (0, 0, 0)), (64, (0, 0, 1)), (64, (1, 0, 2)),      # keys of the longest tile: its first, a later, its last block
    (64, (0, 2, 0)), (64, (1, 2, 2)),                       # values
    (128, (0, 0, 0)), (128, (1, 0, 2)), (128, (0, 2, 1)),   # a block of one tile of the pair
    (128, (2, 0, 1)), (128, (3, 2, 1)), (128, (2, 2, 0)),   # a pair of tiles: the second's last block, both tiles' first
])
def test_packed_after_an_expired_wait(hooks, d, at):
    """Rows of the block that gave up are right or left as they were; all others are right."""
    import torch
    torch.manual_seed(4)
    lens, Hq = [300, 77], 2
    T = sum(lens)
    q = torch.randn((T, Hq, d), device="cuda").bfloat16()
    k, v = torch.randn((2, T, 1, d), device="cuda").bfloat16()
    cu, st = _ints([0, 300, 377]), _ints([0])
    good, out = torch.empty_like(q), torch.full_like(q, 5.0)

    def run(o):
        rc = hooks.dreamer_attn_packed(q.data_ptr(), Hq * d, k.data_ptr(), d, v.data_ptr(), d, o.data_ptr(), Hq * d,
                                       cu.data_ptr(), 2, T, Hq, 1, d, 1, d ** -0.5, st.data_ptr(), None)
        assert rc == 0
        torch.cuda.synchronize()

    run(good)
    assert st.item() == 0
    hooks.dreamer_test_withhold(*at)
    run(out)
    assert st.item() == TIMEOUT
    left = (out == 5.0).all(-1)
    assert 1 <= int(left.sum()) <= (256 if d == 128 else 128)
    assert torch.equal(out[~left], good[~left])
    st.zero_()
    for _ in range(3):                                   # tensor memory was given back
        run(out)
    assert st.item() == 0 and torch.equal(out, good)
