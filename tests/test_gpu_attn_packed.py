"""Causal attention over packed prompts on the GPU against a plain 64-bit reference."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

EPS = {"fp32": 2.0 ** -24, "bf16": 2.0 ** -8}


def _t(x, dtype):
    import torch
    return torch.from_numpy(np.asarray(x, np.float32)).cuda().to(torch.float32 if dtype == "fp32" else torch.bfloat16)


def _f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _ints(v):
    import torch
    return torch.tensor(list(v), dtype=torch.int32, device="cuda")


def reference(q, k, v, cu, scale, dtype):
    """(output, tolerance) in 64 bits; NaN where no prompt writes.

    The tolerance counts, with u = 2^-23 (float32) and eps half a step of the stored type:
      eps |o|             the stored output
      2^-8 sum w |v|      bfloat16 only: the weights as they enter the output product
      2 E sum w |v|       scores off by E = (d + 2) u scale max sum |q||k|, their scaling and the
                          exponential (2^-21 + u |z|), on the weights and on their sum
      (n + 16) u sum w |v|   sums over n keys of weights and of products"""
    T, Hq, d = q.shape
    G = Hq // k.shape[1]
    out = np.full(q.shape, np.nan)
    tol = np.zeros(q.shape)
    u = 2.0 ** -23
    for a, e in zip(cu[:-1], cu[1:]):
        n = e - a
        if n == 0:
            continue
        for h in range(Hq):
            qq, kk, vv = q[a:e, h], k[a:e, h // G], v[a:e, h // G]
            with np.errstate(invalid="ignore", over="ignore"):
                z = qq @ kk.T * scale
                z = np.where(np.arange(n)[None, :] > np.arange(n)[:, None], -np.inf, z)
                m = z.max(1, keepdims=True)
                w = np.exp(z - m)
                w /= w.sum(1, keepdims=True)
            hid = np.arange(n)[None, :] > np.arange(n)[:, None]
            w = np.where(hid, 0.0, w)
            clean = np.isfinite(vv).all()
            if clean:
                o = w @ vv
                av = w @ np.abs(vv)
            else:  # what a row does not see does not reach it
                o, av = np.zeros((n, d)), np.zeros((n, d))
                with np.errstate(invalid="ignore"):
                    for i in range(n):
                        o[i] = w[i, :i + 1] @ vv[:i + 1]
                        av[i] = w[i, :i + 1] @ np.abs(vv[:i + 1])
            out[a:e, h] = o
            with np.errstate(invalid="ignore"):
                az = np.where(hid, 0.0, np.abs(qq) @ np.abs(kk).T).max(1, keepdims=True)
                gap = np.where(hid, 0.0, np.abs(z - m)).max(1, keepdims=True)
                E = (d + 2) * u * scale * az + 2.0 ** -21 + u * (1 + gap)
                tol[a:e, h] = EPS[dtype] * np.abs(o) + (2 * E + (n + 16) * u + (2.0 ** -8 if dtype == "bf16" else 0)) * av
    return out, tol


def _check(got, want, tol, written):
    g, w = got[written], want[written]
    nan = np.isnan(w)
    assert np.array_equal(np.isnan(g), nan)
    err = np.abs(g - w)[~nan]
    assert (err <= tol[written][~nan]).all(), (err / np.maximum(tol[written][~nan], 1e-300)).max()


def _qkv(rng, T, Hq, Hk, d, dtype):
    return (_t(rng.standard_normal((T, Hq, d)) * 1.5, dtype), _t(rng.standard_normal((T, Hk, d)), dtype),
            _t(rng.standard_normal((T, Hk, d)) + rng.standard_normal(d), dtype))


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("fp32", 16), ("fp32", 32), ("fp32", 64), ("fp32", 128)])
@pytest.mark.parametrize("lens,Hq,Hk", [
    ([1], 1, 1),
    ([1, 1, 1], 2, 1),
    ([127, 128, 129], 2, 2),
    ([255, 0, 256, 257, 3], 2, 1),
    ([0, 0, 31, 32, 33, 0], 6, 2),
    ([385, 700], 4, 1),
    ([5] * 70, 1, 1),                        # more prompts than a warp has lanes
])
def test_packed_against_64_bits(cuda, dtype, d, lens, Hq, Hk):
    from depth_recurrent_attention_b200.attention import attn_packed
    rng = np.random.default_rng(sum(lens) + d + Hq)
    q, k, v = _qkv(rng, sum(lens), Hq, Hk, d, dtype)
    cu = np.concatenate([[0], np.cumsum(lens)])
    out = attn_packed(q, k, v, _ints(cu))
    want, tol = reference(_f64(q), _f64(k), _f64(v), cu, d ** -0.5, dtype)
    _check(_f64(out), want, tol, np.ones(sum(lens), bool))


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("fp32", 32)])
@pytest.mark.parametrize("n,longest,first", [(64, 9, 0), (65, 9, 0), (65, 300, 150), (1100, 4, 1), (3000, 2, 700)])
def test_many_prompts(cuda, dtype, d, n, longest, first):
    """As many prompts as change how a block finds its item, empty ones among them, rows of no prompt
    before and behind them."""
    import torch
    from depth_recurrent_attention_b200.attention import attn_packed
    rng = np.random.default_rng(n + longest)
    lens = rng.integers(0, longest + 1, n)
    cu = first + np.concatenate([[0], np.cumsum(lens)])
    T = int(cu[-1]) + 5
    q, k, v = _qkv(rng, T, 2, 1, d, dtype)
    out, st = torch.full_like(q, 3.0), _ints([0])
    attn_packed(q, k, v, _ints(cu), out=out, status=st)
    want, tol = reference(_f64(q), _f64(k), _f64(v), cu, d ** -0.5, dtype)
    written = np.zeros(T, bool)
    written[first:T - 5] = True
    _check(_f64(out), want, tol, written)
    assert (out[~torch.from_numpy(written).cuda()] == 3).all() and st.item() == 0
    bad = cu.copy()
    bad[n // 2] = cu[-1] + 9                     # past the rows, and decreasing behind
    attn_packed(q, k, v, _ints(bad), out=out, status=st)
    assert st.item() != 0 and (out[:first] == 3).all()


@pytest.mark.parametrize("d", [16, 32, 64, 128])
@pytest.mark.parametrize("Hq", [2, 24])       # few items with long rows, and many: two ways to share a row's keys
def test_float32_of_few_and_of_many_items(cuda, Hq, d):
    import torch
    from depth_recurrent_attention_b200.attention import attn_packed
    lens = [257, 1, 480]
    rng = np.random.default_rng(Hq + d)
    q, k, v = _qkv(rng, sum(lens), Hq, 2, d, "fp32")
    cu = [0, 257, 258, 738]
    out = attn_packed(q, k, v, _ints(cu))
    want, tol = reference(_f64(q), _f64(k), _f64(v), cu, d ** -0.5, "fp32")
    _check(_f64(out), want, tol, np.ones(sum(lens), bool))
    assert torch.equal(out, attn_packed(q, k, v, _ints(cu)))
    for r, bad in ((40, np.inf), (300, np.nan), (257 + 1 + 190, -np.inf)):
        v[r, 1, 3] = bad
    want, tol = reference(_f64(q), _f64(k), _f64(v), cu, d ** -0.5, "fp32")
    got, fin = _f64(attn_packed(q, k, v, _ints(cu))), np.isfinite(want)
    assert np.array_equal(np.isfinite(got), fin)
    assert (np.abs(got - want)[fin] <= tol[fin]).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_strides_scale_and_rows_of_no_prompt(cuda, dtype):
    """q, k, v as slices of one fused projection, a given scale, rows before the first and behind
    the last prompt left as they were, and not used whatever they hold."""
    import torch
    from depth_recurrent_attention_b200.attention import attn_packed
    rng = np.random.default_rng(3)
    T, d = 300, 64
    fused = _t(rng.standard_normal((T, 8, d)), dtype)
    cu = [7, 150, 150, 281]
    q, k, v = fused[:, :4], fused[:, 4:6], fused[:, 6:]
    fused[:7, 4:] = float("nan")
    fused[281:, 4:] = float("inf")
    wide = torch.full((T, 6, d), 5.0, dtype=q.dtype, device="cuda")
    out = wide[:, 1:5]
    attn_packed(q, k, v, _ints(cu), out=out, scale=0.3)
    want, tol = reference(_f64(q), _f64(k), _f64(v), cu, float(np.float32(0.3)), dtype)
    written = np.zeros(T, bool)
    written[7:281] = True
    _check(_f64(out), want, tol, written)
    assert (wide[~torch.from_numpy(written).cuda()] == 5).all()
    assert (wide[:, 0] == 5).all() and (wide[:, 5] == 5).all()
    # the same bits with clean surroundings
    clean = fused.clone()
    clean[:7], clean[281:] = 0, 0
    again = attn_packed(clean[:, :4], clean[:, 4:6], clean[:, 6:], _ints(cu), scale=0.3)
    assert torch.equal(again[7:281], out[7:281])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_values_that_are_not_finite_reach_only_the_rows_that_see_them(cuda, dtype, bad):
    """A value that is not finite at row r of a prompt changes the rows from r on, in its key
    head and channel, and no row before it, also inside the same tile; nor another prompt."""
    import torch
    from depth_recurrent_attention_b200.attention import attn_packed
    rng = np.random.default_rng(4)
    lens = [200, 140, 77]
    cu = [0, 200, 340, 417]
    q, k, v = _qkv(rng, 417, 2, 2, 64, dtype)
    base = attn_packed(q, k, v, _ints(cu))
    v2 = v.clone()
    v2[130, 0, 5] = bad      # second tile of the first prompt
    v2[200 + 20, 1, 63] = bad  # first tile of the second
    v2[340, 0, 0] = bad      # first row of the third
    out = attn_packed(q, k, v2, _ints(cu))
    want, tol = reference(_f64(q), _f64(k), _f64(v2), cu, 64 ** -0.5, dtype)
    g = _f64(out)
    fin = np.isfinite(want)
    assert np.array_equal(np.isfinite(g), fin)
    if np.isinf(bad):
        assert np.array_equal(g[~fin], want[~fin])
    assert (np.abs(g - want)[fin] <= tol[fin]).all()
    assert torch.equal(out[:130], base[:130]) and torch.equal(out[200:220], base[200:220])
    k2 = k.clone()
    k2[150, 0, 3] = bad
    ko = attn_packed(q, k2, v, _ints(cu))
    assert torch.equal(ko[:150], base[:150]) and torch.equal(ko[200:], base[200:])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_scores_far_apart(cuda, dtype):
    """Scores that grow by far more than the rescaling threshold along a row, both ways."""
    from depth_recurrent_attention_b200.attention import attn_packed
    rng = np.random.default_rng(8)
    T, d = 600, 64
    q, k, v = _qkv(rng, T, 2, 1, d, dtype)
    q[:] = q.abs()
    ramp = _t(np.linspace(-6, 6, T)[:, None, None] * np.ones((T, 1, d)), dtype)
    for kk in (ramp, ramp.flip(0)):
        out = attn_packed(q, kk, v, _ints([0, T]))
        want, tol = reference(_f64(q), _f64(kk), _f64(v), [0, T], d ** -0.5, dtype)
        _check(_f64(out), want, tol, np.ones(T, bool))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_repeatable_streams_graphs_and_bad_boundaries(cuda, dtype):
    import torch
    from depth_recurrent_attention_b200.attention import attn_packed
    rng = np.random.default_rng(9)
    q, k, v = _qkv(rng, 400, 4, 2, 64, dtype)
    cu = _ints([0, 150, 400])
    a = attn_packed(q, k, v, cu)
    assert torch.equal(attn_packed(q, k, v, cu), a)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = attn_packed(q, k, v, cu, stream=s)
    s.synchronize()
    assert torch.equal(a, b)
    g = torch.cuda.CUDAGraph()
    out = torch.empty_like(a)
    c = cu.clone()
    with torch.cuda.graph(g):
        attn_packed(q, k, v, c, out=out)
    for cut in ([0, 150, 400], [0, 1, 400], [0, 400, 400]):
        c.copy_(_ints(cut))
        g.replay()
        assert torch.equal(out, attn_packed(q, k, v, _ints(cut)))
    # boundaries out of order or outside the rows: reported, nothing outside is touched
    st = _ints([0])
    attn_packed(q, k, v, cu, status=st)
    assert st.item() == 0
    for bad in ([0, 300, 200], [-5, 100, 400], [0, 100, 401], [0, 2 ** 31 - 1, 400]):
        st.zero_()
        attn_packed(q, k, v, _ints(bad), status=st)
        assert st.item() != 0
    # no prompts, or no rows in any
    o = torch.full_like(a, 3.0)
    attn_packed(q, k, v, _ints([0]), out=o)
    attn_packed(q, k, v, _ints([9, 9, 9]), out=o)
    assert (o == 3).all()


def test_two_streams_at_once(cuda):
    import torch
    from depth_recurrent_attention_b200.attention import attn_packed
    rng = np.random.default_rng(10)
    sets = [_qkv(rng, 900, 4, 2, 128, "bf16") for _ in range(2)]
    cu = _ints([0, 333, 900])
    want = [attn_packed(*x, cu) for x in sets]
    torch.cuda.synchronize()
    ss = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(5):
        got = [attn_packed(*x, cu, stream=s) for x, s in zip(sets, ss)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
