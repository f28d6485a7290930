"""Attention over the 4-bit cache where magnitudes lie far apart: the error of bfloat16 calls stays that of
storing the output, whatever the queries look like."""
import numpy as np
import pytest

import kv4_ref as R

pytestmark = pytest.mark.gpu


def _ints(v):
    import torch
    return torch.tensor(list(v), dtype=torch.int32, device="cuda")


def _bf16(x):
    import torch
    return torch.from_numpy(np.asarray(x, np.float32)).cuda().bfloat16()


def _f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _reference(data, d, q, lens, scale):
    """(output, sqrt(sum_j w_j^2 v_j^2), largest s qi) in 64 bits: qi a query's 16-bit step times the scale
    in log2, s a key's."""
    codes, s, m = R.unpack(data, d)
    B, Hq, _ = q.shape
    G = Hq // data.shape[1]
    out, spread, moved = np.zeros(q.shape), np.zeros(q.shape), 0.0
    for b in range(B):
        n = int(lens[b])
        for h in range(Hq):
            k, v = (codes[i, b, h // G, :n] * s[i, b, h // G, :n, :, None] + m[i, b, h // G, :n, :, None]
                    for i in range(2))
            z = k.reshape(n, d) @ q[b, h] * scale
            w = np.exp(z - z.max())
            w /= w.sum()
            out[b, h] = w @ v.reshape(n, d)
            spread[b, h] = np.sqrt(w ** 2 @ v.reshape(n, d) ** 2)
            step = np.abs(q[b, h]).reshape(-1, 64).max(-1) / 32512
            moved = max(moved, (s[0, b, h // G, :n] * step).max() * scale / np.log(2.0))
    return out, spread, moved


@pytest.mark.parametrize("lens,H,G,d,capacity", [
    ([64, 50, 7], 4, 1, 64, 64),
    ([300, 64], 4, 2, 128, 300),
    ([200, 200], 2, 4, 64, 200),
    ([90, 130], 2, 11, 128, 130),
    ([700, 64, 64, 64], 2, 3, 64, 13000),          # runs over all items
    ([90, 500, 64], 2, 8, 128, 13000),
])
@pytest.mark.parametrize("kind", ["ordinary", "one channel 30", "one channel 1000", "half the channels 300", "large", "small scale"])
def test_queries_of_any_spread(cuda, kind, lens, H, G, d, capacity):
    """Relative L2 against 64 bits.  Storing the output is off by half a step of 2^-8 |o| at most, evenly
    distributed: 2^-8 / sqrt(3) at most in root mean square.  A weight is off by E: rounding the queries moves a
    score by 2^-10 at most in root mean square in log2, or by 20 s qi / 254 where the queries have three bytes;
    moved independently, the output is off by E sqrt(sum w^2 v^2), of which three are allowed."""
    from depth_recurrent_attention_b200.attention import KV4Cache
    rng = np.random.default_rng(len(kind) * 1000 + sum(lens) + G)
    T, B = sum(lens), len(lens)
    k, v = rng.standard_normal((2, T, H, d))
    q = rng.standard_normal((B, H * G, d))
    scale = d ** -0.5
    if kind.startswith("one channel"):
        q[:, :, 5] = float(kind.split()[-1]) * rng.choice([-1, 1], (B, H * G))
        k[:, :, 5] = 2.0                            # a channel in which the keys agree
    elif kind.startswith("half"):
        q[:, :, ::2] *= 300
        k[:, :, ::2] = rng.choice([-2.0, 2.0], d // 2)
    elif kind == "large":
        q *= 8
    elif kind == "small scale":
        q *= 2.0 ** 20
        scale *= 2.0 ** -20
    c = KV4Cache.alloc(B, H, d, capacity)
    c.store(_bf16(k), _bf16(v), _ints(np.concatenate([[0], np.cumsum(lens)])), _ints([0] * B))
    qt = _bf16(q)
    got = _f64(c.attend(qt, _ints(lens), scale=scale))
    want, spread, moved = _reference(c.data[0].cpu().numpy(), d, _f64(qt), lens, scale)
    E = np.log(2.0) * (2.0 ** -10 + 20 * moved / 254)
    tol = np.sqrt((2.0 ** -16 / 3) * (want ** 2).sum() + (3 * E) ** 2 * (spread ** 2).sum())
    err = np.sqrt(((got - want) ** 2).sum())
    assert err <= tol, (err / np.sqrt((want ** 2).sum()), tol / np.sqrt((want ** 2).sum()), moved * 20)


@pytest.mark.parametrize("capacity", [192, 192 * 70])
@pytest.mark.parametrize("pair", [0x7F7F, 0x7F80, 0x4700])      # a scale and offset of 3.4e38, infinity, 2^15
def test_scales_behind_the_last_key_change_no_bit(cuda, pair, capacity):
    """Whether a block's queries get their third byte is decided by the keys that count."""
    import torch
    from depth_recurrent_attention_b200.attention import KV4Cache
    rng = np.random.default_rng(31)
    lens, d = [70, 64, 1, 0], 128
    c = KV4Cache.alloc(4, 2, d, capacity)
    k, v = rng.standard_normal((2, 520, 2, d))
    c.store(_bf16(k), _bf16(v), _ints(range(0, 521, 130)), _ints([0] * 4))
    q = _bf16(rng.standard_normal((4, 4, d)))
    a = c.attend(q, _ints(lens))
    nb = capacity // 64
    pos = torch.arange(capacity, device="cuda").view(nb, 64)
    pairs = c.data[0].view(4, 2, nb, -1)[..., 4 * 64 * 32:].view(torch.int16).view(4, 2, nb, 4, 64, 2)
    for b, n in enumerate(lens):
        hidden = (pos >= n)[None, :, None, :, None].expand(2, nb, 4, 64, 2)
        pairs[b][hidden] = pair
    same = torch.equal(a, c.attend(q, _ints(lens)))
    assert same
