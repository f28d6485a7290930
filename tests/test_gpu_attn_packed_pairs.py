"""Packed attention at head dim 128, where a block's two query tiles share every key and value block: values
that are not finite on either tile's diagonal."""
import numpy as np
import pytest

from test_gpu_attn_packed import _f64, _ints, _qkv, reference

pytestmark = pytest.mark.gpu

CU = [0, 300, 456, 712, 800]    # 3 tiles (a pair and one), 2 (the second ragged), 2 full, 1 ragged


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("rows", [
    [20],                        # the pair's first tile
    [200],                       # its second
    [20, 200],                   # both
    [127, 128],                  # at their border: a row whose own key is the only one it sees
    [299],                       # the last row of the tile without a partner
    [300, 455],                  # first and last row of a prompt, in a ragged second tile
    [456 + 255, 712, 799],
])
def test_values_that_are_not_finite_at_head_dim_128(cuda, rows, bad):
    import torch
    from depth_recurrent_attention_b200.attention import attn_packed
    rng = np.random.default_rng(40 + rows[0])
    q, k, v = _qkv(rng, CU[-1], 4, 2, 128, "bf16")
    base = attn_packed(q, k, v, _ints(CU))
    for i, r in enumerate(rows):
        v[r, i % 2, 5 + 60 * i] = bad            # either 64-column half, either key head
    out = attn_packed(q, k, v, _ints(CU))
    want, tol = reference(_f64(q), _f64(k), _f64(v), CU, 128 ** -0.5, "bf16")
    g, fin = _f64(out), np.isfinite(want)
    assert np.array_equal(np.isfinite(g), fin)
    if np.isinf(bad):
        assert np.array_equal(g[~fin], want[~fin])
    assert (np.abs(np.where(fin, g, 0) - np.where(fin, want, 0)) <= np.where(fin, tol, np.inf)).all()
    # Tiles before the first bad row's keep their bits.  In its own tile the diagonal block's product is summed
    # in another order: sums of n <= 128 products differ by n 2^-23 sum w |v| (of which tol, held above, counts
    # n + 16), after which storing in bfloat16 may round to the other neighbour.
    for a, e in zip(CU[:-1], CU[1:]):
        first = min([a + (r - a) // 128 * 128 for r in rows if a <= r < e], default=e)
        same = torch.equal(out[a:first], base[a:first])
        assert same, (a, first)
