"""Cases, plain forms and 64-bit references of the attention operators beside the depth step.

prompt   causal attention over packed prompts of different lengths, with grouped heads:
         out[t, h] = sum_{j <= t, same prompt} softmax_j(q[t, h] . k[j, h // G] / sqrt(d)) v[j, h // G]
cache    rows of keys and values quantised into a 4-bit cache as they are written, and read
         back.  A group is 64 consecutive channels of one head of one token:
         s = (max - min) / 15 and m = min, both rounded to bf16; c = round((x - m) / s) in 0..15
         (half to even, c = 0 where s = 0); the value held is s * c + m.
attend   one query token a sequence over its 4-bit cache, with grouped heads; a sequence of
         length 0 gives zeros.

The cache of one depth is [B][H_kv][capacity / 64][block], a block being 64 tokens: K codes
[d / 64][64 tokens][32 bytes] (channel 2i in the low half of byte i), V codes likewise, K
(s, m) pairs [d / 64][64 tokens][2] in bf16, V pairs likewise.
"""
import math

import torch

own = False

BLOCK = 64   # tokens of a cache block
GROUP = 64   # channels that share a scale and an offset

_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
_SIZE = {"bf16": 2, "fp32": 4}


# ---------------------------------------------------------------------------------- cases
def listed():
    return [
        # a few short chat turns, all heads of the small workload: the call's latency
        dict(name="prompt-turns", op="prompt", dtype="bf16", seqs=4, longest=65, even=False,
             heads=8, kv_heads=8, dim=64),
        # the medium workload's eight prompts of up to 2048 tokens, ragged
        dict(name="prompt-batch", op="prompt", dtype="bf16", seqs=8, longest=2048, even=False,
             heads=16, kv_heads=16, dim=64),
        # the large workload's prompt length and head size, keys shared by groups of four heads
        dict(name="prompt-long", op="prompt", dtype="bf16", seqs=3, longest=8192, even=False,
             heads=16, kv_heads=4, dim=128),
        # float32 mode: odd lengths, two heads a key head
        dict(name="prompt-fp32", op="prompt", dtype="fp32", seqs=6, longest=777, even=False,
             heads=4, kv_heads=2, dim=64),
        # the decode workload's append: one new token for each of 64 sequences
        dict(name="cache-append", op="cache", dtype="bf16", seqs=64, longest=1, even=True,
             heads=16, kv_heads=16, dim=64, used=4000),
        # prompts of the large workload written to an empty cache
        dict(name="cache-fill", op="cache", dtype="bf16", seqs=3, longest=8192, even=False,
             heads=16, kv_heads=16, dim=128, used=0),
        # float32 rows of odd lengths behind a partly filled cache
        dict(name="cache-fp32", op="cache", dtype="fp32", seqs=5, longest=513, even=False,
             heads=4, kv_heads=4, dim=128, used=100),
        # a handful of short sequences: the call's latency
        dict(name="attend-short", op="attend", dtype="bf16", seqs=4, longest=300, even=False,
             heads=8, kv_heads=8, dim=64),
        # the decode workload: 64 sequences of 4096 cached tokens, every head its own keys
        dict(name="attend-decode", op="attend", dtype="bf16", seqs=64, longest=4096, even=True,
             heads=16, kv_heads=16, dim=64),
        # ragged sequences up to the large workload's length, four query heads a key head
        dict(name="attend-grouped", op="attend", dtype="bf16", seqs=32, longest=8192, even=False,
             heads=16, kv_heads=4, dim=128),
        # one very long sequence: few rows, a long axis
        dict(name="attend-one-long", op="attend", dtype="bf16", seqs=1, longest=131071, even=True,
             heads=16, kv_heads=4, dim=128),
        # float32 queries over the same kind of cache
        dict(name="attend-fp32", op="attend", dtype="fp32", seqs=8, longest=1000, even=False,
             heads=8, kv_heads=8, dim=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompt", "cache", "attend"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    dim = rng.choice([64, 128])
    kv_heads = rng.choice([1, 2, 4, 8, 16])
    group = rng.choice([g for g in (1, 2, 3, 4, 5, 8) if g * kv_heads <= 16])
    heads = kv_heads * group
    even = rng.random() < 0.25
    if op == "prompt":
        longest = _log(rng, 1, 8192 if dtype == "bf16" else 2048)
        seqs = _log(rng, 1, max(1, min(64, 16384 // longest)))
        return dict(op=op, dtype=dtype, seqs=seqs, longest=longest, even=even, heads=heads,
                    kv_heads=kv_heads, dim=dim)
    if op == "cache":
        longest = _log(rng, 1, 8192)
        seqs = _log(rng, 1, max(1, min(128, 16384 // longest)))
        return dict(op=op, dtype=dtype, seqs=seqs, longest=longest, even=even, heads=kv_heads,
                    kv_heads=kv_heads, dim=dim, used=_log(rng, 1, 2000) - 1)
    tokens = (1 << 27) // (kv_heads * dim)    # half the decode workload's cache at most
    longest = _log(rng, 1, min(131071, tokens))
    seqs = _log(rng, 1, max(1, min(128, tokens // longest)))
    return dict(op=op, dtype=dtype, seqs=seqs, longest=longest, even=even, heads=heads,
                kv_heads=kv_heads, dim=dim)


def _lengths(case):
    """Tokens of each sequence: all the longest, or spread below it, short ones the most."""
    n, top = case["seqs"], case["longest"]
    if case["even"]:
        return [top] * n
    part = [(i * 0.6180339887498949 + 0.37) % 1.0 for i in range(n)]
    return [top if i == 0 else 1 + int((top - 1) * part[i] ** 2) for i in range(n)]


def _capacity(case):
    top = case["longest"] + case.get("used", 0) + 1
    return -(-top // BLOCK) * BLOCK


def work(case):
    lens, d, es = _lengths(case), case["dim"], _SIZE[case["dtype"]]
    hq, hk, total = case["heads"], case["kv_heads"], sum(_lengths(case))
    row4 = hk * (d // 2 + d // GROUP * 4)      # bytes of one token's packed keys (or values)
    if case["op"] == "prompt":
        pairs = sum(n * (n + 1) // 2 for n in lens)
        return {"bytes": es * d * total * (2 * hq + 2 * hk), "flops": 4.0 * hq * d * pairs}
    if case["op"] == "cache":
        # written: rows in, packed rows out; read back: packed rows in, rows out
        return {"bytes": 2 * total * (2 * hk * d * es + 2 * row4), "flops": 8.0 * total * hk * d}
    return {"bytes": 2 * total * row4 + 2 * es * d * hq * case["seqs"],
            "flops": 4.0 * hq * d * total}


# --------------------------------------------------------------------------------- inputs
def _rows(shape, seed, tid, dtype, shift=0.0):
    g = torch.Generator(device="cuda")
    g.manual_seed((seed * 1000003 + tid) % (1 << 62))
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    if shift:  # a mean of its own for each channel, as keys and values have
        x = x + shift * torch.randn(shape[-1], generator=g, device="cuda", dtype=torch.float32)
    return x.to(_DT[dtype])


def _cu(lens):
    return torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).to(torch.int32).cuda()


def _pack(codes, s, m):
    """codes [B][H][N][ng][64] and (s, m) [B][H][N][ng] -> bytes of the code planes and of the
    pairs of every block, N a multiple of 64."""
    B, H, N, ng = s.shape
    byte = (codes[..., 0::2] | (codes[..., 1::2] << 4)).to(torch.uint8)
    byte = byte.view(B, H, N // BLOCK, BLOCK, ng, 32).transpose(3, 4).reshape(B, H, N // BLOCK, -1)
    pair = torch.stack([s, m], -1).to(torch.bfloat16).view(B, H, N // BLOCK, BLOCK, ng, 2)
    pair = pair.transpose(3, 4).contiguous().view(B, H, N // BLOCK, -1).view(torch.uint8)
    return byte, pair


def prepare(case, seed):
    lens, d, dt = _lengths(case), case["dim"], case["dtype"]
    hq, hk, n, total = case["heads"], case["kv_heads"], case["seqs"], sum(_lengths(case))
    st = dict(case)
    if case["op"] == "prompt":
        st.update(q=_rows((total, hq, d), seed, 1, dt), k=_rows((total, hk, d), seed, 2, dt),
                  v=_rows((total, hk, d), seed, 3, dt, 0.3), cu=_cu(lens))
        # rows of every prompt in a padded batch, as the plain form needs them
        st["lens"] = torch.tensor(lens, dtype=torch.int64).cuda()
        return st
    cap, ng = _capacity(case), d // GROUP
    bytes_ = 2 * ng * BLOCK * (32 + 4)
    if case["op"] == "cache":
        st.update(k=_rows((total, hk, d), seed, 1, dt, 1.0), v=_rows((total, hk, d), seed, 2, dt, 0.3),
                  cu=_cu(lens), start=torch.full((n,), case["used"], dtype=torch.int32).cuda(),
                  data=torch.zeros((1, n, hk, cap // BLOCK, bytes_), dtype=torch.uint8, device="cuda"))
        return st
    parts = []
    for tid, shift in ((1, 1.0), (2, 0.3)):
        parts.append(_pack(*_quantise(_rows((n, hk, cap, d), seed, tid, "bf16", shift))))
    (kb, kp), (vb, vp) = parts
    st.update(data=torch.cat([kb, vb, kp, vp], -1).unsqueeze(0).contiguous(),
              q=_rows((n, hq, d), seed, 3, dt),
              lens=torch.tensor(lens, dtype=torch.int32).cuda())
    return st


# ---------------------------------------------------------------------------- plain forms
def _quantise(x):
    """Codes and (s, m) of rows x [..., d]: [..., d / 64, 64] and [..., d / 64] twice.  The
    step and the quotients are taken in 64 bits: a quotient next to a half must not move."""
    x = x.reshape(*x.shape[:-1], x.shape[-1] // GROUP, GROUP)
    hi, lo = x.amax(-1).double(), x.amin(-1).double()
    s = ((hi - lo) / 15.0).float().bfloat16().double()
    m = lo.float().bfloat16().double()
    c = torch.round((x.double() - m[..., None]) / torch.where(s > 0, s, 1.0)[..., None])
    c = torch.where(s[..., None] > 0, c.clamp(0, 15), 0.0)
    return c.to(torch.int32), s.float(), m.float()


def _values(st):
    """Keys and values held in the cache, in 32 bits: [B][H][capacity][d] twice."""
    data, ng = st["data"][0], st["dim"] // GROUP
    B, H, nb, _ = data.shape
    out, at = [], ng * BLOCK * 32
    for i in range(2):
        byte = data[..., i * at:(i + 1) * at].reshape(B, H, nb, ng, BLOCK, 32)
        pair = data[..., 2 * at + i * ng * BLOCK * 4:2 * at + (i + 1) * ng * BLOCK * 4]
        pair = pair.contiguous().view(torch.bfloat16).float().view(B, H, nb, ng, BLOCK, 2)
        c = torch.stack([byte & 15, byte >> 4], -1).float().flatten(-2)
        x = c * pair[..., :1] + pair[..., 1:]
        out.append(x.transpose(3, 4).reshape(B, H, nb * BLOCK, ng * GROUP))
    return out


def _prompt(st):
    lens, G = st["lens"], st["heads"] // st["kv_heads"]
    top, n = st["longest"], st["seqs"]
    pos = torch.arange(top, device="cuda")
    real = pos[None, :] < lens[:, None]
    at = torch.where(real, st["cu"][:-1, None].long() + pos, 0)
    q = st["q"][at].transpose(1, 2).float()                       # [n][Hq][top][d]
    k = st["k"][at].transpose(1, 2).float().repeat_interleave(G, 1)
    v = st["v"][at].transpose(1, 2).float().repeat_interleave(G, 1)
    z = torch.matmul(q, k.transpose(2, 3)) / math.sqrt(st["dim"])
    z.masked_fill_(pos[None, :] > pos[:, None], -math.inf)
    z -= z.amax(-1, keepdim=True)
    z.exp_()
    z /= z.sum(-1, keepdim=True)
    o = torch.matmul(z, v)
    return o.transpose(1, 2)[real].to(st["q"].dtype)


def _held(x):
    c, s, m = _quantise(x)
    return (c.float() * s[..., None] + m[..., None]).flatten(-2).to(x.dtype)


def _attend(st):
    k, v = _values(st)
    B, H, cap, d = k.shape
    q = st["q"].float().view(B, H, st["heads"] // H, d)
    z = torch.matmul(q, k.transpose(2, 3)) / math.sqrt(d)
    hidden = torch.arange(cap, device="cuda")[None, :] >= st["lens"][:, None]
    z.masked_fill_(hidden[:, None, None, :], -math.inf)
    p = torch.exp(z - z.amax(-1, keepdim=True).clamp_min(-3e38))
    o = torch.matmul(p, v) / p.sum(-1, keepdim=True).clamp_min(1e-30)
    return o.reshape(B, st["heads"], d).to(st["q"].dtype)


def run(state):
    st = state
    if own:
        from depth_recurrent_attention_b200 import attention
        if st["op"] == "prompt":
            return attention.attn_packed(st["q"], st["k"], st["v"], st["cu"])
        cache = attention.KV4Cache(st["data"], st["dim"])
        if st["op"] == "cache":
            cache.store(st["k"], st["v"], st["cu"], st["start"])
            return cache.load(st["cu"], st["start"], st["k"].shape[0], st["k"].dtype)
        return cache.attend(st["q"], st["lens"])
    if st["op"] == "prompt":
        return _prompt(st)
    if st["op"] == "cache":
        return _held(st["k"]), _held(st["v"])
    return _attend(st)


# ------------------------------------------------------------------------------ 64 bits
def _softmax_rows(q, k, v, first):
    """softmax(q k^T / sqrt(d)) v in 64 bits; row i sees the keys up to first + i."""
    z = (q @ k.T) / math.sqrt(q.shape[1])
    i = torch.arange(q.shape[0], device=q.device)[:, None] + first
    z = z.masked_fill(torch.arange(k.shape[0], device=q.device)[None, :] > i, -math.inf)
    return torch.softmax(z, 1) @ v


def exact(case, seed):
    st = prepare(case, seed)
    lens, d = _lengths(case), case["dim"]
    G = case["heads"] // case["kv_heads"]
    if case["op"] == "prompt":
        out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
        at = 0
        for n in lens:
            for h in range(case["heads"]):
                k = st["k"][at:at + n, h // G].double()
                v = st["v"][at:at + n, h // G].double()
                for r in range(0, n, 4096):
                    e = min(n, r + 4096)
                    out[at + r:at + e, h] = _softmax_rows(
                        st["q"][at + r:at + e, h].double(), k[:e], v[:e], r)
            at += n
        return out
    if case["op"] == "cache":
        out = []
        for x in (st["k"], st["v"]):
            y = x.double().unflatten(-1, (-1, GROUP))
            low = y.min(-1, keepdim=True).values
            step = (y.max(-1, keepdim=True).values - low) / torch.tensor(15.0, dtype=torch.float64, device="cuda")
            step, low = step.to(torch.bfloat16).double(), low.to(torch.bfloat16).double()
            c = torch.where(step > 0, (y - low) / step, torch.zeros_like(y))
            out.append((c.round().clip(0, 15) * step + low).flatten(-2))
        return tuple(out)
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    plane = BLOCK * 32
    ng = d // GROUP
    for b, n in enumerate(lens):
        blocks = st["data"][0, b, :, :-(-n // BLOCK)]
        kv = []
        for side in range(2):
            x = torch.empty((blocks.shape[0], blocks.shape[1] * BLOCK, d), dtype=torch.float64, device="cuda")
            for g in range(ng):
                code = blocks[:, :, (side * ng + g) * plane:(side * ng + g + 1) * plane]
                code = code.reshape(blocks.shape[0], -1, 32).int()
                p0 = 2 * ng * plane + (side * ng + g) * BLOCK * 4
                pair = blocks[:, :, p0:p0 + BLOCK * 4].contiguous().view(torch.bfloat16).double()
                pair = pair.reshape(blocks.shape[0], -1, 2)
                x[:, :, g * GROUP:(g + 1) * GROUP:2] = (code % 16) * pair[..., :1] + pair[..., 1:]
                x[:, :, g * GROUP + 1:(g + 1) * GROUP:2] = (code // 16) * pair[..., :1] + pair[..., 1:]
            kv.append(x[:, :n])
        for h in range(case["heads"]):
            out[b, h] = _softmax_rows(st["q"][b, h:h + 1].double(), kv[0][h // G], kv[1][h // G], n - 1)[0]
    return out
