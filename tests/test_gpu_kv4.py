"""The 4-bit cache on the GPU against a plain 64-bit reference: rows stored and read back, the
bytes of the cache, and single-token attention over it."""
import numpy as np
import pytest

import kv4_ref as R

pytestmark = pytest.mark.gpu


def _t(x, dtype):
    import torch
    return torch.from_numpy(np.asarray(x, np.float32)).cuda().to(torch.float32 if dtype == "fp32" else torch.bfloat16)


def _f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _ints(v):
    import torch
    return torch.tensor(list(v), dtype=torch.int32, device="cuda")


EPS = {"fp32": 2.0 ** -24, "bf16": 2.0 ** -8}


def _case(rng, lens, H, d, dtype):
    T = sum(lens)
    k = rng.standard_normal((T, H, d)) + rng.standard_normal(d) * 2
    v = rng.standard_normal((T, H, d)) * np.exp(rng.standard_normal((T, H, 1)))
    return _t(k, dtype), _t(v, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("lens,start,H,d", [
    ([1], [0], 1, 64),
    ([1, 1, 1, 1, 1], [0, 63, 64, 127, 5], 3, 64),      # one row a sequence: a decode step
    ([5, 0, 130, 64], [0, 0, 3, 64], 2, 128),           # an empty sequence, block borders
    ([0, 0, 17], [0, 0, 60], 5, 64),
    ([33, 70], [1, 50], 9, 128),                         # more (head, plane) pairs than a CTA's eight
])
def test_store_writes_the_format_and_nothing_else(cuda, dtype, lens, start, H, d):
    import torch
    from depth_recurrent_attention_b200.attention import KV4Cache
    rng = np.random.default_rng(len(lens) * 100 + H)
    k, v = _case(rng, lens, H, d, dtype)
    cap = 256
    c = KV4Cache.alloc(len(lens), H, d, cap)
    c.data.random_(0, 256)
    before = c.data[0].cpu().numpy().copy()
    cu = np.concatenate([[0], np.cumsum(lens)])
    c.store(k, v, _ints(cu), _ints(start))
    codes, s, m = R.unpack(c.data[0].cpu().numpy(), d)
    c0, s0, m0 = R.unpack(before, d)
    for side, x in enumerate((k, v)):
        rc, rs, rm = R.quantise(_f64(x))
        for b, n in enumerate(lens):
            at = slice(start[b], start[b] + n)
            row = slice(cu[b], cu[b] + n)
            c0[side, b, :, at], s0[side, b, :, at], m0[side, b, :, at] = (
                y[row].swapaxes(0, 1) for y in (rc, rs, rm))
    assert np.array_equal(codes, c0)
    assert np.array_equal(s, s0, equal_nan=True) and np.array_equal(m, m0, equal_nan=True)
    # read back: s c + m rounded once
    for out in (torch.float32, torch.bfloat16):
        ks, vs = c.load(_ints(cu), _ints(start), sum(lens), out)
        for x, y in ((k, ks), (v, vs)):
            want = R.held(_f64(x))
            want = R.bf16(want) if out == torch.bfloat16 else want.astype(np.float32).astype(np.float64)
            assert np.array_equal(_f64(y), want)


def test_quotients_next_to_a_half_and_constant_groups(cuda):
    """Values on every border between two codes, one float32 step to each side of it, constant
    groups, tiny and huge ranges: the codes are those of exact arithmetic."""
    from depth_recurrent_attention_b200.attention import KV4Cache
    rng = np.random.default_rng(5)
    rows = []
    for s in (1.0, 0.3330078125, 2.0 ** -100, 3e-39, 1e28, 7.0):
        s = float(R.bf16([s])[0])
        x = np.float32(s) * (rng.integers(0, 15, 64) + 0.5).astype(np.float32)
        x = np.nextafter(x, np.where(np.arange(64) % 3 == 0, np.inf, np.where(np.arange(64) % 3 == 1, -np.inf, x)).astype(np.float32))
        x[0], x[1] = 0.0, np.float32(15 * s)
        rows.append(x)
        rows.append(np.full(64, np.float32(s)))
    rows.append(np.zeros(64, np.float32))
    rows.append(np.where(np.arange(64) == 9, 1e-45, 0).astype(np.float32))
    x = np.stack(rows)[:, None]
    n = len(rows)
    k = _t(x, "fp32")
    v = _t(-x, "fp32")
    c = KV4Cache.alloc(1, 1, 64, n)
    c.store(k, v, _ints([0, n]), _ints([0]))
    codes, s, m = R.unpack(c.data[0].cpu().numpy(), 64)
    for side, y in enumerate((k, v)):
        rc, rs, rm = R.quantise(_f64(y))
        assert np.array_equal(s[side, 0, 0, :n, 0], rs[:, 0, 0]) and np.array_equal(m[side, 0, 0, :n, 0], rm[:, 0, 0])
        assert np.array_equal(codes[side, 0, 0, :n, 0], rc[:, 0, 0])


def test_groups_that_are_not_finite_read_back_as_nan_and_stay_alone(cuda):
    import torch
    from depth_recurrent_attention_b200.attention import KV4Cache
    rng = np.random.default_rng(6)
    x = rng.standard_normal((6, 2, 128)).astype(np.float32)
    x[1, 0, 70] = np.nan
    x[2, 1, 3] = np.inf
    x[3, 1, 127] = -np.inf
    x[4, 0, 0] = 3e38
    c = KV4Cache.alloc(1, 2, 128, 64)
    c.store(_t(x, "fp32"), _t(x, "fp32"), _ints([0, 6]), _ints([0]))
    k, v = c.load(_ints([0, 6]), _ints([0]), 6, torch.float32)
    want = R.held(x.astype(np.float64))
    assert np.isnan(want).sum() == 4 * 64
    for y in (k, v):
        assert np.array_equal(_f64(y), want.astype(np.float32).astype(np.float64), equal_nan=True)


def test_rows_of_no_sequence_and_positions_outside_the_cache(cuda):
    """Rows before the first and behind the last boundary, and positions outside the cache, are
    neither stored nor loaded; the latter set the status."""
    import torch
    from depth_recurrent_attention_b200.attention import KV4Cache
    rng = np.random.default_rng(7)
    x = _t(rng.standard_normal((40, 2, 64)), "bf16")
    c = KV4Cache.alloc(2, 2, 64, 64)
    st = _ints([0])
    c.store(x, x, _ints([3, 10, 20]), _ints([0, 30]), status=st)
    assert st.item() == 0
    data = c.data.clone()
    codes, s, _ = R.unpack(data[0].cpu().numpy(), 64)
    assert (s[:, 0, :, :7] != 0).all() and (s[:, 0, :, 7:] == 0).all()
    assert (s[:, 1, :, 30:40] != 0).all() and (s[:, 1, :, :30] == 0).all() and (s[:, 1, :, 40:] == 0).all()
    c.store(x, x, _ints([0, 0, 10]), _ints([0, 60]), status=st)   # positions 64.. are outside
    assert st.item() != 0
    st.zero_()
    c.store(x, x, _ints([0, 4, 4]), _ints([-4, 0]), status=st)    # negative positions
    assert st.item() != 0
    assert torch.equal(c.data[0, 0], data[0, 0])
    out = (torch.full((40, 2, 64), 7.0, device="cuda"), torch.full((40, 2, 64), 7.0, device="cuda"))
    st.zero_()
    k, v = c.load(_ints([3, 10, 20]), _ints([0, 60]), 40, torch.float32, out=out, status=st)
    assert st.item() != 0
    for y in (k, v):
        left = torch.ones(40, dtype=torch.bool)
        left[3:14] = False                             # 10..13 are positions 60..63
        assert (y[left.cuda()] == 7.0).all() and (y[3:14] != 7.0).any(-1).all()
    k, v = c.load(_ints([3, 10, 20]), _ints([0, 60]), 40, torch.float32)
    assert (k[left.cuda()] == 0).all()


def _cache(rng, lens, H, d, cap, dtype="bf16"):
    from depth_recurrent_attention_b200.attention import KV4Cache
    c = KV4Cache.alloc(len(lens), H, d, cap)
    k, v = _case(rng, lens, H, d, dtype)
    if sum(lens):
        c.store(k, v, _ints(np.concatenate([[0], np.cumsum(lens)])), _ints([0] * len(lens)))
    return c


@pytest.mark.parametrize("capacity", [0, 13000])   # as much as is needed; enough for runs over all items
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("lens,H,G,d", [
    ([1], 1, 1, 64),
    ([0, 1, 2, 63, 64, 65, 129], 2, 1, 64),             # empty, single keys, block borders
    ([200, 17], 2, 2, 128),
    ([77, 300], 1, 3, 64),                              # a head count between two forms
    ([40, 513], 2, 4, 128),
    ([90, 1], 1, 5, 128),
    ([260], 1, 8, 64),
    ([100, 31], 1, 11, 64),                             # two chunks of query heads
    ([3000, 1500], 1, 1, 128),                          # split over a cluster
    ([5000], 1, 2, 64),
])
def test_attend_against_64_bits(cuda, dtype, lens, H, G, d, capacity):
    rng = np.random.default_rng(sum(lens) + H * G)
    c = _cache(rng, lens, H, d, max(capacity, max(lens) + 1))
    q = _t(rng.standard_normal((len(lens), H * G, d)) * 2, dtype)
    out = c.attend(q, _ints(lens))
    ref, tol = R.attend(c.data[0].cpu().numpy(), d, _f64(q), lens, d ** -0.5, EPS[dtype])
    err = np.abs(_f64(out) - ref)
    assert (err <= tol).all(), (err / np.maximum(tol, 1e-300)).max()


@pytest.mark.parametrize("dtype,small", [("bf16", -110), ("fp32", -100)])
def test_attend_of_small_numbers(cuda, dtype, small):
    """Queries and values near the least normal numbers count as others do: queries of 2^-112 over keys
    of 2^98, values of 2^-110 (float32: 2^-100, whose third bfloat16 term is a normal number)."""
    from depth_recurrent_attention_b200.attention import KV4Cache
    rng = np.random.default_rng(21)
    k, v = rng.standard_normal((2, 40, 2, 64))
    c = KV4Cache.alloc(1, 2, 64, 64)
    c.store(_t(k * 2.0 ** 97, dtype), _t(v * 2.0 ** small, dtype), _ints([0, 40]), _ints([0]))
    q = _t(rng.standard_normal((1, 4, 64)) * 2.0 ** (small - 3), dtype)
    scale = 2.0 ** (-97 - small)
    out = c.attend(q, _ints([40]), scale=scale)
    ref, tol = R.attend(c.data[0].cpu().numpy(), 64, _f64(q), [40], scale, EPS[dtype], floor=2.0 ** -110)
    err = np.abs(_f64(out) - ref)
    assert (err <= tol).all(), (err / tol).max()
    assert (tol.max(-1) < np.abs(ref).max(-1) / 4).all()


@pytest.mark.parametrize("capacity", [192, 192 * 70])
def test_attend_does_not_use_what_lies_behind_the_last_key(cuda, capacity):
    """NaN pairs and random codes behind lens[b] change no bit."""
    import torch
    rng = np.random.default_rng(11)
    lens = [70, 64, 1, 0]
    c = _cache(rng, [130] * 4, 2, 128, capacity)
    q = _t(rng.standard_normal((4, 4, 128)), "bf16")
    a = c.attend(q, _ints(lens))
    nb = capacity // 64
    pos = torch.arange(capacity, device="cuda").view(nb, 64)
    plane = c.data[0].view(4, 2, nb, -1)
    pairs = plane[..., 4 * 64 * 32:].view(torch.int16).view(4, 2, nb, 4, 64, 2)
    for b, n in enumerate(lens):
        hid = (pos >= n)[None, :, None, :, None].expand(2, nb, 4, 64, 2)
        pairs[b][hid] = 0x7FC0
    b_ = c.attend(q, _ints(lens))
    assert torch.equal(a, b_) and (b_[3] == 0).all()


def test_attend_of_nan_keys_and_large_scores(cuda):
    """A NaN group among the keys makes its own heads NaN and no others; scores far apart (one
    key takes all the weight) stay exact."""
    import torch
    from depth_recurrent_attention_b200.attention import KV4Cache
    rng = np.random.default_rng(12)
    k = rng.standard_normal((200, 2, 64))
    v = rng.standard_normal((200, 2, 64))
    k[50, 1, 5] = np.nan
    c = KV4Cache.alloc(1, 2, 64, 200)
    c.store(_t(k, "fp32"), _t(v, "fp32"), _ints([0, 200]), _ints([0]))
    q = _t(rng.standard_normal((1, 4, 64)), "fp32")
    o = c.attend(q, _ints([200]))
    assert torch.isfinite(o[0, :2]).all() and torch.isnan(o[0, 2:]).all()
    assert torch.isfinite(c.attend(q, _ints([50]))).all()
    big = c.attend(q * 1e4, _ints([50]))
    ref, tol = R.attend(c.data[0].cpu().numpy(), 64, _f64(q * 1e4), [50], 64 ** -0.5, EPS["fp32"])
    assert (np.abs(_f64(big) - ref) <= tol).all()


@pytest.mark.parametrize("capacity", [2048, 16384])
def test_attend_strides_streams_graphs_and_repeatability(cuda, capacity):
    """q as a slice of a wider row, out in place of q, another stream, a captured and replayed
    graph whose lengths change between replays: the same bits as the plain call."""
    import torch
    rng = np.random.default_rng(13)
    lens = [2000, 700, 64]
    c = _cache(rng, lens, 2, 64, capacity)
    wide = _t(rng.standard_normal((3, 12, 64)), "bf16")
    q = wide[:, 4:8]
    ln = _ints(lens)
    a = c.attend(q.contiguous(), ln)
    assert torch.equal(c.attend(q, ln), a) and torch.equal(c.attend(q, ln), a)
    own = wide.clone()
    c.attend(own[:, 4:8], ln, out=own[:, 4:8])
    assert torch.equal(own[:, 4:8], a) and torch.equal(own[:, :4], wide[:, :4]) and torch.equal(own[:, 8:], wide[:, 8:])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = c.attend(q, ln, stream=s)
    s.synchronize()
    assert torch.equal(b, a)
    g = torch.cuda.CUDAGraph()
    out = torch.empty_like(a)
    with torch.cuda.graph(g):
        c.attend(q, ln, out=out)
    for cut in ([2000, 700, 64], [1, 0, 33]):
        ln.copy_(_ints(cut))
        g.replay()
        assert torch.equal(out, c.attend(q, _ints(cut)))


@pytest.mark.parametrize("capacity", [64, 64 * 200])
def test_attend_reports_lengths_outside_the_cache(cuda, capacity):
    import torch
    rng = np.random.default_rng(14)
    c = _cache(rng, [60, 60], 1, 64, capacity)
    q = _t(rng.standard_normal((2, 1, 64)), "bf16")
    st = _ints([0])
    good = c.attend(q, _ints([60, 64]), status=st)
    assert st.item() == 0
    for bad in (capacity + 1, -1, 2 ** 31 - 1):
        st.zero_()
        o = c.attend(q, _ints([60, bad]), status=st)
        assert st.item() != 0 and torch.equal(o[0], good[0]) and (o[1] == 0).all()


def test_offsets_past_32_bits(cuda):
    """A cache of more than 2^32 bytes: the last depth's last sequence is its own."""
    import torch
    from depth_recurrent_attention_b200.attention import KV4Cache
    rng = np.random.default_rng(15)
    c = KV4Cache(torch.empty((1, 4, 2, 62 * 1024, 9216), dtype=torch.uint8, device="cuda"), 128)
    assert c.data.numel() > 2 ** 32
    n = 300
    at = c.capacity - n
    k, v = _case(rng, [n], 2, 128, "bf16")
    cu = _ints([0, 0, 0, 0, n])
    c.store(k, v, cu, _ints([0, 0, 0, at]))
    a, b = c.load(cu, _ints([0, 0, 0, at]), n, torch.float32)
    assert np.array_equal(_f64(a), R.held(_f64(k))) and np.array_equal(_f64(b), R.held(_f64(v)))


def test_attend_over_many_items_and_long_runs(cuda):
    """More query heads than a chunk, sequences from none to several CTAs' runs: each head equals the
    same head attended with the others' sequences emptied (the runs then lie elsewhere) to rounding."""
    import torch
    rng = np.random.default_rng(16)
    lens = [0, 12800, 1, 7000, 0, 65, 300, 9999]
    c = _cache(rng, lens, 2, 128, 12800)
    q = _t(rng.standard_normal((8, 22, 128)), "fp32")
    a = c.attend(q, _ints(lens))
    assert (a[0] == 0).all() and (a[4] == 0).all()
    for b in (1, 3, 5, 7):
        only = [n if i == b else 0 for i, n in enumerate(lens)]
        o = c.attend(q, _ints(only))
        # the order of float32 sums over n keys: n 2^-23 of the sum of magnitudes, here below 64 |v|
        assert (o[b] - a[b]).abs().max() <= lens[b] * 2.0 ** -23 * 64
        assert (o[[i for i in range(8) if i != b]] == 0).all()


def test_two_streams_attend_at_once(cuda):
    """Each call has a workspace of its own."""
    import torch
    rng = np.random.default_rng(17)
    cs = [_cache(rng, [9000, 100], 2, 64, 13000) for _ in range(2)]
    q = _t(rng.standard_normal((2, 4, 64)), "bf16")
    ln = _ints([9000, 100])
    want = [c.attend(q, ln) for c in cs]
    torch.cuda.synchronize()
    ss = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = [c.attend(q, ln, stream=s) for c, s in zip(cs, ss)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
