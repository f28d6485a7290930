"""The handle's packed prefill and its decode over 4-bit caches on the GPU: prompts of different
lengths against the oracle's forward of each prompt alone, every depth of a decode step against
its own normalised states in 64 bits, and the way from prompts to tokens."""
import numpy as np
import pytest

import kv4_ref as R
import oracle as O
import parity as PY
from depth_recurrent_attention_b200 import configs, inputs

pytestmark = pytest.mark.gpu


def _handle(cfg, W, **kw):
    from depth_recurrent_attention_b200.dreamer import Dreamer
    return Dreamer(cfg, {k: inputs.to_device(v, "fp32" if k == "bias" else cfg.dtype) for k, v in W.items()}, **kw)


def _ints(v):
    import torch
    return torch.tensor(list(v), dtype=torch.int32, device="cuda")


def _trace(cfg, n, names):
    import torch
    dt = torch.float32 if cfg.dtype == "fp32" else torch.bfloat16
    L, h, k = cfg.depth, cfg.hidden, cfg.top_k
    make = dict(y=((L, n, h), dt), xhat=((L, n, h), dt), sa_k=((L, n, h), dt), sa_v=((L, n, h), dt),
                y_f32=((L, n, h), torch.float32), x_f32=((L, n, h), torch.float32),
                idx=((L, n, k), torch.int32), w=((L, n, k), torch.float32),
                pidx=((L, n), torch.int32), psig=((L, n), torch.float32))
    return {f: torch.zeros(make[f][0], dtype=make[f][1], device="cuda") for f in names}


# one expert for every slot (E = k) and at most one projection expert: no routing decision can
# flip, so bf16 runs stay comparable through every depth
FREE = dict(n_experts=4, top_k=4)


@pytest.mark.parametrize("base,lens,kw", [
    ("tiny", [5, 1, 0, 9], {}),
    ("tiny", [16], dict(variant=1)),
    ("tiny", [3, 4, 2], dict(variant=2)),
    ("tiny", [7, 8], dict(variant=3)),
    ("small", [1, 129, 0, 200, 77], dict(depth=3, **FREE)),
    ("small", [300, 100], dict(depth=3, n_proj_experts=1, **FREE)),          # grouped projections
    ("small", [130, 2, 250], dict(depth=2, n_heads=4, head_dim=128, **FREE)),
    ("small", [150, 77], dict(depth=2, variant=1, n_proj_experts=1, **FREE)),  # serial layout, rows gathered
    ("small", [150, 77], dict(depth=2, variant=2, **FREE)),
    ("small", [150, 77], dict(depth=2, variant=3, n_proj_experts=1, **FREE)),
    ("small", [150, 77], dict(depth=3, da_window=2, **FREE)),
    ("small", [1], dict(depth=2, **FREE)),
    ("small", [64, 65], dict(depth=2, dtype="fp32", n_experts=16, top_k=2)),
])
def test_packed_forward_equals_each_prompt_alone(cuda, base, lens, kw):
    import torch
    cfg = configs.CONFIGS[base].with_(**kw)
    if base == "tiny":
        cfg = cfg.with_(batch=2, seq=16)
    T = sum(lens)
    W = inputs.host_weights(cfg)
    dev = _handle(cfg, W)
    x0 = inputs.extra_normal(cfg, 5001, (T, cfg.hidden), 1.0)
    cu = np.concatenate([[0], np.cumsum(lens)])
    tr = _trace(cfg, T, ["y", "y_f32", "x_f32", "idx", "sa_k", "sa_v"])
    out = dev.forward_packed(inputs.to_device(x0, cfg.dtype), _ints(cu), trace=tr)
    counts = dev.route_counts().numpy()
    assert (counts.sum(1) == T * cfg.top_k).all()
    bf = cfg.dtype == "bf16"
    D = PY.deployed_weights(cfg, W)
    for a, e in zip(cu[:-1], cu[1:]):
        if a == e:
            continue
        one = cfg.with_(batch=1, seq=int(e - a))
        r = O.Oracle(one, D).forward(x0[a:e])
        for l in range(cfg.depth):
            if not bf:
                _, flips = PY.check_routing(one, W, l, tr["idx"][l, a:e].cpu().numpy(), r["idx"][l],
                                            r["margin"][l], strict=True)
                assert flips == 0
            # The serial layout's sequence attention reads u = x^ + DA W_O rounded to bf16, half a step of
            # 2^-8 |u|.  With projection experts the absorbed weights have twice the variance, |u| reaches
            # 8 and its rounding 2^-6 = 1.6e-2 an element; W_QKV and W_O (each of gain sqrt 2 in rms) double
            # that to 3.1e-2 before any other rounding: the absolute bound of 3e-2 says nothing there, for
            # the equal-length forward as little (its states are the same bits, below).
            loose = cfg.variant == 1 and cfg.n_proj_experts > 0
            PY.check_drift(PY.to_np(tr["y"][l, a:e]), r["y"][l], f"y depth {l} rows {a}..{e}",
                           gate_abs=l == 0 and bf and not loose, f32=PY.to_np(tr["y_f32"][l, a:e]))
            PY.check_drift(PY.to_np(tr["sa_k"][l, a:e]), r["sa_k"][l], f"k depth {l}", gate_abs=False)
            PY.check_drift(PY.to_np(tr["sa_v"][l, a:e]), r["sa_v"][l], f"v depth {l}", gate_abs=False)
        if bf:
            PY.check_drift(PY.to_np(out[a:e]), r["x_out"], "x_out", False, f32=PY.to_np(tr["x_f32"][-1, a:e]))
        else:
            PY.check_hidden(PY.to_np(out[a:e]), r["x_out"], False, "x_out")
    # run again without the trace: directly, captured into a graph, replayed
    x = inputs.to_device(x0, cfg.dtype)
    c, o = _ints(cu), torch.empty_like(out)
    for _ in range(4):
        o.zero_()
        dev.forward_packed(x, c, x_out=o)
        assert torch.equal(o, out)
    dev.close()


@pytest.mark.parametrize("kw", [dict(), dict(variant=1), dict(variant=1, n_proj_experts=1), dict(variant=2),
                                dict(variant=3), dict(n_proj_experts=1), dict(n_heads=4, head_dim=128)])
def test_packed_equal_prompts_are_the_equal_length_forward(cuda, kw):
    import torch
    cfg = configs.SMALL.with_(batch=2, seq=256, depth=2, **{**FREE, **kw})
    W = inputs.host_weights(cfg)
    dev = _handle(cfg, W)
    x = inputs.to_device(inputs.extra_normal(cfg, 5003, (cfg.tokens, cfg.hidden), 1.0), "bf16")
    a = {n: t for n, t in _trace(cfg, cfg.tokens, ["y_f32"]).items()}
    b = {n: t for n, t in _trace(cfg, cfg.tokens, ["y_f32"]).items()}
    dev.forward(x, trace=a)
    dev.forward_packed(x, _ints([0, 256, 512]), trace=b)
    # the same arithmetic in the same order but for the sums inside the attention kernels
    assert PY.rel_l2(PY.to_np(b["y_f32"][0]), PY.to_np(a["y_f32"][0])) <= 1e-3
    dev.close()


def test_packed_forward_with_projection_experts_one_depth(cuda):
    """Several projection experts: rows in group order, outputs at their sorted rows."""
    cfg = configs.SMALL.with_(depth=1, n_proj_experts=8, n_experts=4, top_k=4)
    lens = [200, 1, 333, 64]
    T = sum(lens)
    W = inputs.host_weights(cfg)
    dev = _handle(cfg, W)
    x0 = inputs.extra_normal(cfg, 5002, (T, cfg.hidden), 1.0)
    cu = np.concatenate([[0], np.cumsum(lens)])
    tr = _trace(cfg, T, ["y", "y_f32", "xhat", "pidx", "psig"])
    dev.forward_packed(inputs.to_device(x0, "bf16"), _ints(cu), trace=tr)
    D = PY.deployed_weights(cfg, W)
    for a, e in zip(cu[:-1], cu[1:]):
        one = cfg.with_(batch=1, seq=int(e - a))
        r = O.Oracle(one, D).forward(x0[a:e])
        gp = tr["pidx"][0, a:e].cpu().numpy()
        # a token with another projection expert changes the rows after it too: none may differ
        assert PY.proj_same_as_forward(one, W, 0, gp, r["pidx"][0], r["pmargin"][0],
                                       PY.to_np(tr["xhat"][0, a:e]), r["xhat"][0]).all()
        PY.check_hidden(PY.to_np(tr["y"][0, a:e]), r["y"][0], True, f"y rows {a}..{e}",
                        f32=PY.to_np(tr["y_f32"][0, a:e]))
    dev.close()


def _caches(cfg, lens, seed):
    """4-bit caches of random past tokens for every depth."""
    from depth_recurrent_attention_b200.attention import KV4Cache
    c = KV4Cache.alloc(cfg.batch, cfg.n_heads, cfg.head_dim, cfg.cache_len + 1, depth=cfg.depth)
    cu, zero = _ints(np.concatenate([[0], np.cumsum(lens)])), _ints([0] * cfg.batch)
    for l in range(cfg.depth):
        shape = (sum(lens), cfg.n_heads, cfg.head_dim)
        k = inputs.to_device(inputs.extra_normal(cfg, seed + 2 * l, shape, 1.0), cfg.dtype)
        v = inputs.to_device(inputs.extra_normal(cfg, seed + 2 * l + 1, shape, 1.0), cfg.dtype)
        if sum(lens):
            c.store(k, v, cu, zero, depth=l)
    return c


@pytest.mark.parametrize("lens,kw", [
    ([300, 1, 77, 0], dict(variant=3)),
    ([300, 1, 77, 0], dict(da_window=1)),
    ([64, 63], dict(da_window=1, n_heads=4, head_dim=128)),
    ([0], dict(da_window=1)),
    ([130, 64, 5], dict(variant=3, dtype="fp32")),
    ([130, 64, 5], dict(da_window=1, dtype="fp32", n_heads=4, head_dim=128)),
    ([(7 * i) % 61 for i in range(70)], dict(da_window=1)),
    ([40, 0, 17], dict(da_window=1, n_proj_experts=1)),
    ([13000, 5], dict(variant=3, depth=1)),               # long caches: runs over all items
])
def test_decode_step_over_4_bit_caches(cuda, lens, kw):
    """Every depth against its own x^ (traced): the new key and value are in the cache within half
    a step, and y = x^ + W_O [SA over what the cache holds | DA], where a window of one depth makes
    DA the depth's own value."""
    import torch
    cfg = configs.SMALL.with_(**{**dict(batch=len(lens), seq=1, depth=3, cache_len=max(lens) + 1), **FREE, **kw})
    B, h, d, H = cfg.batch, cfg.hidden, cfg.head_dim, cfg.n_heads
    W = inputs.host_weights(cfg)
    dev = _handle(cfg, W)
    c = _caches(cfg, lens, 6001)
    before = c.data.clone()
    x = inputs.to_device(inputs.extra_normal(cfg, 6100, (B, h), 1.0), cfg.dtype)
    ln = _ints(lens)
    tr = _trace(cfg, B, ["xhat", "y", "y_f32"] + (["psig"] if cfg.n_proj_experts else []))
    out = dev.decode_step_kv4(x, c, ln, trace=tr)
    dev.route_counts()                                   # no device error
    assert torch.isfinite(out).all()
    bf = cfg.dtype == "bf16"
    D = PY.deployed_weights(cfg, W)
    wq, wo = D["w_qkv"][0].astype(np.float64), D["w_o"][0].astype(np.float64)
    for l in range(cfg.depth):
        xh = PY.to_np(tr["xhat"][l])
        sig = PY.to_np(tr["psig"][l])[:, None] if cfg.n_proj_experts else 1.0   # one projection expert
        qkv = sig * (xh @ wq)
        q, k, v = (qkv[:, i * h:(i + 1) * h].reshape(B, H, d) for i in range(3))
        q = np.stack([[O.rope(q[b, j], lens[b]) for j in range(H)] for b in range(B)])
        k = np.stack([[O.rope(k[b, j], lens[b]) for j in range(H)] for b in range(B)])
        kk, vv = c.load(_ints(range(B + 1)), ln, B, torch.float32, depth=l)
        for want, got in ((k, PY.to_np(kk)), (v, PY.to_np(vv))):
            g = want.reshape(B, H, -1, 64)
            step = (g.max(-1) - g.min(-1)) / 15
            # half a step, the scale's rounding over 15 steps, the row's storage and offset in bf16
            tol = (0.5 + 15 * 2.0 ** -8) * step + 2.0 ** -7 * np.abs(g).max(-1) + 1e-4
            assert (np.abs(got.reshape(g.shape) - g) <= tol[..., None]).all()
        att, _ = R.attend(c.data[l].cpu().numpy(), d, q, [n + 1 for n in lens], d ** -0.5, 0.0)
        da = qkv[:, 5 * h:] if cfg.variant != 3 else np.zeros((B, h))
        y = xh + sig * (np.concatenate([att.reshape(B, h), da], 1) @ wo)
        PY.check_hidden(PY.to_np(tr["y"][l]), y, bf, f"y depth {l}", f32=PY.to_np(tr["y_f32"][l]) if bf else None)
    # nothing but the new positions changed
    pos = torch.arange(c.capacity, device="cuda")
    new, old = c.data, before
    for l in range(cfg.depth):
        n_codes, n_s, n_m = R.unpack(new[l].cpu().numpy(), d)
        o_codes, o_s, o_m = R.unpack(old[l].cpu().numpy(), d)
        for b, n in enumerate(lens):
            keep = np.arange(c.capacity) != n
            assert np.array_equal(n_codes[:, b][:, :, keep], o_codes[:, b][:, :, keep])
            assert np.array_equal(n_s[:, b][:, :, keep], o_s[:, b][:, :, keep])
    # again without the trace: directly, captured into a graph, replayed
    o2 = torch.empty_like(out)
    for _ in range(4):
        o2.zero_()
        dev.decode_step_kv4(x, c, ln, x_out=o2)
        assert torch.equal(o2, out)
    dev.close()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_from_packed_prompts_to_tokens(cuda, dtype):
    """Packed prefill, the prompts' keys and values into the 4-bit caches, three decode steps: the
    caches hold what prefill traced, and each step attends one token more."""
    import torch
    from depth_recurrent_attention_b200.attention import KV4Cache
    lens = [150, 1, 40, 64]
    cfg = configs.SMALL.with_(batch=4, seq=128, depth=2, cache_len=0, dtype=dtype, **FREE)
    T = sum(lens)
    W = inputs.host_weights(cfg)
    dev = _handle(cfg, W, max_cache_len=160)
    cu, zero = _ints(np.concatenate([[0], np.cumsum(lens)])), _ints([0] * 4)
    tr = _trace(cfg, T, ["sa_k", "sa_v"])
    x = inputs.to_device(inputs.extra_normal(cfg, 7001, (T, cfg.hidden), 1.0), dtype)
    dev.forward_packed(x, cu, trace=tr)
    c = KV4Cache.alloc(4, cfg.n_heads, cfg.head_dim, 160, depth=cfg.depth)
    for l in range(cfg.depth):
        rows = [tr[n][l].view(T, cfg.n_heads, cfg.head_dim) for n in ("sa_k", "sa_v")]
        c.store(*rows, cu, zero, depth=l)
        for got, want in zip(c.load(cu, zero, T, torch.float32, depth=l), rows):
            assert np.array_equal(PY.to_np(got), R.held(PY.to_np(want)).astype(np.float32))
    ln = _ints(lens)
    for step in range(3):
        xs = inputs.to_device(inputs.extra_normal(cfg, 7100 + step, (4, cfg.hidden), 1.0), dtype)
        out = dev.decode_step_kv4(xs, c, ln)
        assert torch.isfinite(out).all()
        assert (dev.route_counts().sum(1) == 4 * cfg.top_k).all()
        k, v = c.load(_ints(range(5)), ln, 4, torch.float32)
        assert (k != 0).any(-1).all() and (v != 0).any(-1).all()
        ln += 1
    # a position past max_cache_len is reported by the next call
    from depth_recurrent_attention_b200.dreamer import ERR_ARG, DreamerError
    dev.decode_step_kv4(xs, c, _ints([160, 0, 0, 0]))
    with pytest.raises(DreamerError) as e:
        dev.route_counts()
    assert e.value.code == ERR_ARG
    dev.close()


def test_refusals(cuda):
    import torch
    from depth_recurrent_attention_b200.attention import KV4Cache
    from depth_recurrent_attention_b200.dreamer import ERR_ARG, ERR_STATE, ERR_UNSUPPORTED, DreamerError
    cfg = configs.SMALL.with_(batch=2, seq=64, depth=2, **FREE)
    W = inputs.host_weights(cfg)
    dev = _handle(cfg, W)
    x = inputs.to_device(inputs.extra_normal(cfg, 1, (200, cfg.hidden), 1.0), "bf16")

    def refused(code, fn, *a, **kw):
        with pytest.raises(DreamerError) as e:
            fn(*a, **kw)
        assert e.value.code == code

    refused(ERR_UNSUPPORTED, dev.forward, x[:128])                        # equal prompts of 64: not a multiple of 128
    dev.forward_packed(x[:128], _ints([0, 64, 128]))
    refused(ERR_ARG, dev.forward_packed, x[:129], _ints([0, 129]))        # more than batch * seq
    refused(ERR_ARG, dev.forward_packed, x[:0], _ints([0, 0]))
    refused(ERR_ARG, dev.forward_packed, x[:8], _ints([0]))
    refused(ERR_ARG, dev.forward_packed, x[:8], _ints([0, 8]), depth_begin=1)
    with pytest.raises(ValueError):
        dev.forward_packed(x[:8], torch.tensor([0, 8], device="cuda"))
    for bad in ([0, 5], [1, 8], [0, 6, 5, 8], [0, 9, 8]):                  # reported by the next call
        dev.forward_packed(x[:8], _ints(bad))
        refused(ERR_ARG, dev.route_counts)
    dev.forward_packed(x[:100], _ints([0, 100]))                          # longer than seq + 1 positions
    refused(ERR_ARG, dev.route_counts)
    dev.forward_packed(x[:65], _ints([0, 65]))
    dev.route_counts()
    c = KV4Cache.alloc(2, 8, 64, 128, depth=2)
    refused(ERR_STATE, dev.decode_step_kv4, x[:2], c, _ints([0, 0]))      # a handle without a cache
    dev.close()
    dev = _handle(cfg, W, max_cache_len=129)
    refused(ERR_ARG, dev.decode_step_kv4, x[:2], c, _ints([0, 0]))        # a smaller cache
    refused(ERR_ARG, dev.decode_step_kv4, x[:2], KV4Cache.alloc(3, 8, 64, 192, depth=2), _ints([0, 0]))
    refused(ERR_ARG, dev.decode_step_kv4, x[:2], KV4Cache.alloc(2, 4, 128, 192, depth=2), _ints([0, 0]))
    with pytest.raises(ValueError):
        dev.decode_step_kv4(x[:2], KV4Cache.alloc(2, 8, 64, 192, depth=1), _ints([0, 0]))
    dev.close()


def test_tensors_that_the_binding_refuses(cuda):
    import torch
    from depth_recurrent_attention_b200.attention import KV4Cache
    cfg = configs.SMALL.with_(batch=2, seq=64, depth=2, **FREE)
    dev = _handle(cfg, inputs.host_weights(cfg), max_cache_len=64)
    x = inputs.to_device(inputs.extra_normal(cfg, 1, (16, cfg.hidden), 1.0), "bf16")
    cu, c, lens = _ints([0, 8]), KV4Cache.alloc(2, 8, 64, 64, depth=2), _ints([0, 3])
    for bad in (x[:8].float(), x[:8].cpu(), x[:8, :64], x[::2], x[:8].view(-1), x[:8, :64].contiguous()):
        for kw in (dict(x_in=bad), dict(x_in=x[:8], x_out=bad)):
            with pytest.raises(ValueError):
                dev.forward_packed(cu_seqlens=cu, **kw)
    with pytest.raises(ValueError):
        dev.forward_packed(x[:8], cu, x_out=x[:9].clone())
    for bad in (cu.long(), cu.cpu(), cu.view(1, 2), _ints([0, 0, 8, 8])[::2]):
        with pytest.raises(ValueError):
            dev.forward_packed(x[:8], bad)
    for bad in (x[:1], x[:3], x[:2].float(), x[:2].cpu(), x[:4:2]):
        for kw in (dict(x_new=bad), dict(x_new=x[:2], x_out=bad)):
            with pytest.raises(ValueError):
                dev.decode_step_kv4(cache=c, cache_len=lens, **kw)
    for bad in (lens.long(), lens.cpu(), lens[:1], _ints([0, 0, 0])):
        with pytest.raises(ValueError):
            dev.decode_step_kv4(x[:2], c, bad)
    assert not c.data.any()
    dev.close()
