"""A plain 64-bit reference of the 4-bit cache: numpy, written from the format alone.

A group is 64 channels: s = (max - min) / 15 and m = min, both rounded to bf16 (through
float32), c = rint((x - m) / s) in 0..15 (0 where s = 0), value s c + m; a group with a NaN or a
magnitude above 2^100 holds NaN.  A block is 64 tokens: K codes [ng][64][32 bytes] (channel 2i
low), V codes, K pairs [ng][64][2] bf16, V pairs.
"""
import numpy as np

from depth_recurrent_attention_b200.inputs import bf16_bits_to_f32, f32_to_bf16_bits

BLOCK, GROUP = 64, 64


def bf16(x):
    with np.errstate(over="ignore", invalid="ignore"):
        x32 = np.asarray(x, np.float64).astype(np.float32)
    bits = f32_to_bf16_bits(x32)
    bits = np.where(np.isnan(x32), np.uint16(0x7FC0), bits)
    return bf16_bits_to_f32(bits).astype(np.float64)


def quantise(x):
    """x [..., d] float64 -> (codes [..., ng, 64] int, s, m [..., ng] float64)."""
    x = np.asarray(x, np.float64)
    x = x.reshape(*x.shape[:-1], x.shape[-1] // GROUP, GROUP)
    bad = ~(np.abs(x) <= 2.0 ** 100).all(-1)
    x = np.where(bad[..., None], 0.0, x)
    s = bf16((x.max(-1) - x.min(-1)) / 15.0)
    m = bf16(x.min(-1))
    q = np.rint((x - m[..., None]) / np.where(s > 0, s, 1.0)[..., None])
    c = np.where(s[..., None] > 0, np.clip(q, 0, 15), 0).astype(np.int64)
    nan = np.where(bad, np.nan, 0.0)
    return c, s + nan, m + nan


def held(x):
    c, s, m = quantise(x)
    v = c * s[..., None] + m[..., None]
    return v.reshape(*v.shape[:-2], -1)


def unpack(data, d):
    """data uint8 [B][H][nb][bytes] -> (codes [2][B][H][nb * 64][ng][64], s, m [2][B][H][nb * 64][ng])."""
    B, H, nb, _ = data.shape
    ng = d // GROUP
    codes, s, m = [], [], []
    for side in range(2):
        at = side * ng * BLOCK * 32
        by = data[..., at:at + ng * BLOCK * 32].reshape(B, H, nb, ng, BLOCK, 32).astype(np.int64)
        c = np.empty((B, H, nb, ng, BLOCK, 64), np.int64)
        c[..., 0::2] = by & 15
        c[..., 1::2] = by >> 4
        codes.append(c.transpose(0, 1, 2, 4, 3, 5).reshape(B, H, nb * BLOCK, ng, 64))
        at = 2 * ng * BLOCK * 32 + side * ng * BLOCK * 4
        pr = np.ascontiguousarray(data[..., at:at + ng * BLOCK * 4]).view(np.uint16)
        pr = bf16_bits_to_f32(pr.reshape(B, H, nb, ng, BLOCK, 2)).astype(np.float64)
        pr = pr.transpose(0, 1, 2, 4, 3, 5).reshape(B, H, nb * BLOCK, ng, 2)
        s.append(pr[..., 0])
        m.append(pr[..., 1])
    return np.stack(codes), np.stack(s), np.stack(m)


def attend(data, d, q, lens, scale, out_eps, floor=2.0 ** -102):
    """(output, tolerance) [B][Hq][d] of one query token a sequence.

    The tolerance counts, per element, with unit roundoffs u = 2^-23 (float32, either rounding
    mode) and out_eps (half a step of the output type):
      out_eps |o|                       the stored output
      out_eps sum_j w_j s_j |c_j - 8|   float32: the weights w_j s_j as they enter the output product in
                                        three bf16 terms (2^-24)
      2 E sum_j w_j |v_j|               scores off by E = (d + 8) u scale (sum |q||s (c - 8)| +
                                        |m + 8 s| sum |q|) at most over the keys, times log 2 rounding
                                        and the exponential (2^-21), on weights and on their sum
      n u sum_j w_j |v_j|               the sums over n keys, of weights and of products
    bfloat16 (out_eps 2^-8) scores are taken with q in steps of its plane's largest |q| / 32512: each
    q is off by half a step at most, so E has scale sum over planes of (half a step) sum s c more.
    Its weights w_j s_j are taken in steps of the largest of a block of 64 keys / 65535: sum over
    blocks of half a step times sum c.  Neither step is below that of a largest of 2^-110; weights are
    relative to a maximum that is at most 2^8 behind, so w_j s_j count from `floor` = 2^-102 on, and from
    2^-110 on where there is one block.
    """
    codes, s, m = unpack(data, d)
    B, Hq, _ = q.shape
    H = data.shape[1]
    G = Hq // H
    out, tol = np.zeros((B, Hq, d)), np.zeros((B, Hq, d))
    u = 2.0 ** -23
    for b in range(B):
        n = int(lens[b])
        if n == 0:
            continue
        for h in range(Hq):
            kc, ks, km = codes[0, b, h // G, :n], s[0, b, h // G, :n], m[0, b, h // G, :n]
            vc, vs, vm = codes[1, b, h // G, :n], s[1, b, h // G, :n], m[1, b, h // G, :n]
            k = (kc * ks[..., None] + km[..., None]).reshape(n, d)
            v = (vc * vs[..., None] + vm[..., None]).reshape(n, d)
            qq = np.asarray(q[b, h], np.float64)
            z = k @ qq * scale
            w = np.exp(z - z.max())
            w /= w.sum()
            o = w @ v
            aq = np.abs(qq).reshape(-1, 64)
            e = (np.abs(kc - 8) * ks[..., None] * aq).sum((1, 2)) + (np.abs(km + 8 * ks) * aq.sum(-1)).sum(1)
            if out_eps == 2.0 ** -8:
                e = e + (np.maximum(aq.max(-1), 2.0 ** -110) / 65024 * (kc * ks[..., None]).sum(-1)).sum(-1) / ((d + 8) * u)
            E = (d + 8) * u * abs(scale) * e.max() + 2.0 ** -21 + u * (1 + np.abs(z - z.max()).max())
            absv = w @ np.abs(v) + w @ (np.abs(vm + 8 * vs)[..., None] + np.zeros((1, 1, 64))).reshape(n, d)
            spread = w @ (np.abs(vc - 8) * vs[..., None]).reshape(n, d)
            out[b, h] = o
            if out_eps == 2.0 ** -8:
                spread = np.zeros(d)
                for j in range(0, n, 64):
                    step = np.maximum((w[j:j + 64, None] * vs[j:j + 64]).max(0), floor) / 65535   # [ng]
                    spread += (step[:, None] / 2 * vc[j:j + 64].sum(0)).reshape(d)
                tol[b, h] = out_eps * np.abs(o) + spread
            else:
                tol[b, h] = out_eps * np.abs(o) + out_eps * spread
            tol[b, h] += (2 * E + (n + 16) * u) * absv
    return out, tol
