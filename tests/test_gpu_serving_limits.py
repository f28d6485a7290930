"""Positions and states that the serving paths refuse: what they leave alone."""
import pytest

from depth_recurrent_attention_b200 import configs, inputs

pytestmark = pytest.mark.gpu


def _ints(v):
    import torch
    return torch.tensor(list(v), dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("capacity", [160, 13000])        # 160: rounded up to 192; 13000: the split form
def test_a_refused_decode_position_changes_nothing_in_the_cache(cuda, dtype, capacity):
    """A position from max_cache_len up to the cache's capacity is refused as the dense step refuses it: the
    sequence's cache keeps its bytes at every depth, the others' tokens are stored."""
    import torch
    from depth_recurrent_attention_b200.attention import KV4Cache
    from depth_recurrent_attention_b200.dreamer import ERR_ARG, Dreamer, DreamerError
    cfg = configs.SMALL.with_(batch=3, seq=64, depth=2, cache_len=0, dtype=dtype, n_experts=4, top_k=4)
    W = inputs.host_weights(cfg)
    dev = Dreamer(cfg, {k: inputs.to_device(v, "fp32" if k == "bias" else cfg.dtype) for k, v in W.items()},
                  max_cache_len=160)
    c = KV4Cache.alloc(3, cfg.n_heads, cfg.head_dim, capacity, depth=cfg.depth)
    assert c.capacity > 160
    c.data.random_(0, 60)                                    # small finite pairs
    x = inputs.to_device(inputs.extra_normal(cfg, 7200, (3, cfg.hidden), 1.0), dtype)
    before = c.data.clone()
    good = dev.decode_step_kv4(x, c, _ints([5, 159, 7]))
    dev.route_counts()
    stored = c.data.clone()
    same = torch.equal(stored[:, 1], before[:, 1])
    assert not same
    for bad in (160, c.capacity - 1, c.capacity, -1, 2 ** 31 - 1):
        c.data.copy_(before)
        out = dev.decode_step_kv4(x, c, _ints([5, bad, 7]))
        with pytest.raises(DreamerError) as e:
            dev.route_counts()
        assert e.value.code == ERR_ARG
        same = torch.equal(c.data[:, 1], before[:, 1])
        assert same, bad
        same = torch.equal(c.data[:, 0], stored[:, 0]) and torch.equal(c.data[:, 2], stored[:, 2])
        assert same, bad
        same = torch.equal(out[0], good[0]) and torch.equal(out[2], good[2])
        assert same, bad
    dev.close()


def test_decode_without_programmatic_launches(cuda, monkeypatch):
    """DREAMER_NO_PDL and stage profiling launch every kernel after the one before has ended: the same bits."""
    import torch
    from depth_recurrent_attention_b200.attention import KV4Cache
    from depth_recurrent_attention_b200.dreamer import Dreamer
    cfg = configs.SMALL.with_(batch=2, seq=64, depth=2, cache_len=0, n_experts=4, top_k=4)
    W = {k: inputs.to_device(v, "fp32" if k == "bias" else cfg.dtype) for k, v in inputs.host_weights(cfg).items()}
    x = inputs.to_device(inputs.extra_normal(cfg, 7300, (2, cfg.hidden), 1.0), cfg.dtype)
    lens = _ints([12000, 70])                                   # the split form and its join
    data = torch.randint(0, 60, (2, 2, 8, 13056 // 64, 4608), dtype=torch.uint8, device="cuda")

    def step(profile=False):
        dev = Dreamer(cfg, W, max_cache_len=13000)
        if profile:
            dev.set_profiling(True)
        c = KV4Cache(data.clone(), 64)
        out = [dev.decode_step_kv4(x, c, lens).clone() for _ in range(3)]
        dev.route_counts()
        dev.close()
        return out

    want = step()
    got = step(profile=True)
    monkeypatch.setenv("DREAMER_NO_PDL", "1")
    for a, b, c in zip(want, got, step()):
        assert torch.equal(a, b) and torch.equal(a, c)
