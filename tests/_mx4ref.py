"""Plain 64-bit numpy reference of the MX element rules, the blocked scale layout, the routed layer and
the grouped product, written from their definitions (no code shared with the package)."""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
E4M3 = np.array([m * 2.0 ** -9 for m in range(8)] +
                [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:119])  # codes 0 .. 0x7E
EMAX = {4: 2, 8: 8}


def table(bits):
    return E2M1 if bits == 4 else E4M3


def encode(x, bits):
    """x [..., C] (float64) -> (codes [..., C] one per element, scale bytes [..., C / 32])."""
    t = table(bits)
    n = t.size
    sign_bit, bad = (8, 7) if bits == 4 else (0x80, 0x7F)
    b = np.asarray(x, dtype=np.float64)
    b = b.reshape(b.shape[:-1] + (b.shape[-1] // 32, 32))
    fin = np.isfinite(b).all(-1)
    amax = np.abs(np.where(fin[..., None], b, 0)).max(-1)
    e = np.where(amax > 0, np.frexp(np.where(amax > 0, amax, 1))[1] - 1 - EMAX[bits], -127)
    e = np.maximum(e, -127)
    a = np.abs(np.where(fin[..., None], b, 0)) * np.ldexp(1.0, -e)[..., None]
    i = np.searchsorted((t[1:] + t[:-1]) / 2, a, side="left")     # ties to the lower code
    j = np.minimum(i + 1, n - 1)
    i = np.where(((t[i] + t[j]) / 2 == a) & (i % 2 == 1), j, i)  # then to the even one
    code = np.where(fin[..., None], i, bad) | np.where(np.signbit(b), sign_bit, 0)
    s = np.where(fin, e + 127, 255)
    return code.reshape(np.shape(x)).astype(np.uint8), s.astype(np.uint8)


def decode(code, s, bits):
    t = table(bits)
    every = np.concatenate([t, -t]) if bits == 4 else np.concatenate([t, [np.nan], -t, [np.nan]])
    v = every[code]
    f = np.where(s == 255, np.nan, np.ldexp(1.0, s.astype(np.int64) - 127))
    return (v.reshape(v.shape[:-1] + (v.shape[-1] // 32, 32)) * f[..., None]).reshape(v.shape)


def mx_value(x, bits):
    return decode(*encode(x, bits), bits)


def pack(code):
    """E2M1 codes, two to a byte, even elements low."""
    return (code[..., 0::2] | (code[..., 1::2] << 4)).astype(np.uint8)


def unpack(q):
    return np.stack([q & 15, q >> 4], -1).reshape(q.shape[:-1] + (-1,))


def tiles(s, ends=None):
    """Scale bytes [R, C] -> the blocked layout's bytes, group by group (None: one group)."""
    R, C = s.shape
    ends = [R] if ends is None else list(ends)
    ct = -(-C // 4)
    out, start = [], 0
    for end in ends:
        n = end - start
        for band in range(-(-n // 128)):
            t = np.zeros((ct, 32, 4, 4), np.uint8)
            for r in range(min(128, n - band * 128)):
                for c in range(C):
                    t[c // 4, r % 32, r // 32, c % 4] = s[start + band * 128 + r, c]
            out.append(t.reshape(-1))
        start = end
    return np.concatenate(out) if out else np.zeros(0, np.uint8)


def silu(x):
    return x / (1 + np.exp(-x))


def route(logits, k, score):
    """Per token: the experts of its k largest logits (NaN above all, ties to the lowest index, -inf never)
    and their weights."""
    out = []
    for l in np.asarray(logits, np.float64):
        key = np.where(np.isnan(l), np.inf, l)
        order = sorted(range(l.size), key=lambda e: (not np.isnan(l[e]), -key[e], e))
        pick = [e for e in order if not l[e] == -np.inf][:k]
        v = l[pick]
        if not pick:
            w = v
        elif score == "sigmoid":
            w = 1 / (1 + np.exp(-v))
        else:
            top = v if score == "softmax" else l
            m = np.max(top)
            w = np.exp(v - m) / np.sum(np.exp(top - m))
        out.append((pick, w))
    return out


def moe(x, logits, k, score, gate, up, down, bits):
    """x [T, D], weights as 64-bit values [E, H, D], [E, H, D], [E, D, H] -> y [T, D]."""
    y = np.zeros(x.shape)
    xq = mx_value(x, bits)
    for t, (pick, w) in enumerate(route(logits, k, score)):
        for e, p in zip(pick, w):
            h = silu(gate[e] @ xq[t]) * (up[e] @ xq[t])
            y[t] += p * (down[e] @ mx_value(h, bits))
    return y
