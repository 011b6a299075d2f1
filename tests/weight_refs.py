"""Few tokens with values of both signs, where the rounding of the softmax weights is what shows, and the bound for
8-bit caches: weights rounded to 11 significant bits (at most 2^-11 of each product) instead of the 8 that
tests/attn_refs.py grants to every format. The other terms are those derived there."""
from __future__ import annotations

import numpy as np
import torch

import attn_refs as R

WEIGHT = 2.0 ** -11


def rounded(x, bits):
    """float64 to `bits` significant bits, to nearest."""
    m, e = np.frexp(x)
    return np.ldexp(np.rint(np.ldexp(m, bits)), e - bits)


def case(seed, fmt, kv, G, d, lens):
    """q [B, kv * G, d], and per sequence K and V code values with their scales, [n, kv, ..] (float64, on the CPU)."""
    r = np.random.default_rng(seed)

    def bf16(x):
        return torch.from_numpy(x).bfloat16().double().numpy()
    q = bf16(r.normal(size=(len(lens), kv * G, d)))
    rows = []
    for n in lens:
        k = R.quantise(bf16(r.normal(size=(n, kv, d))), fmt)
        size = (r.random(size=(n, kv, d)) + 0.5) * np.exp2(r.integers(-6, 6, size=(n, kv, 1)))
        v = R.quantise(bf16(size * r.choice((-1.0, 1.0), size=(n, kv, d))), fmt)
        rows.append((*k, *v))
    return q, rows


def want(q, rows, scale):
    """(out, bound) [B, q_heads, d]: attn_refs.attend, its weight term replaced."""
    H, kv = q.shape[1], rows[0][0].shape[1]
    G = H // kv
    out, bound = (np.zeros(q.shape) for _ in range(2))
    for b, (kc, ks, vc, vs) in enumerate(rows):
        for h in range(kv):
            g = slice(h * G, (h + 1) * G)
            x, k, v = (torch.from_numpy(np.ascontiguousarray(t, dtype=np.float64)) for t in
                       (q[b, g], kc[:, h] * ks[:, h, None].astype(np.float64), vc[:, h] * vs[:, h, None].astype(np.float64)))
            o, _, e = R.attend(x, k, v, scale)
            a, _, _ = R.attend(x, k, v.abs(), scale)
            out[b, g], bound[b, g] = o, e - (R.U - WEIGHT) * a
    return out, bound


def with_weights_of(bits, q, rows, scale):
    """The results of 64-bit attention whose weights times V's scales are rounded to `bits` significant bits, in BF16."""
    H, kv = q.shape[1], rows[0][0].shape[1]
    G = H // kv
    out = np.zeros(q.shape)
    for b, (kc, ks, vc, vs) in enumerate(rows):
        for h in range(kv):
            z = scale * q[b, h * G:(h + 1) * G] @ (kc[:, h] * ks[:, h, None].astype(np.float64)).T
            w = np.exp(z - z.max(1, keepdims=True))
            out[b, h * G:(h + 1) * G] = rounded(w * vs[:, h].astype(np.float64), bits) @ vc[:, h] / w.sum(1, keepdims=True)
    return torch.from_numpy(out).bfloat16().double().numpy()
