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
