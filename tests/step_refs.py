"""Plain 64-bit forms of the rotation, the head norms and the window, with the error bounds that the GPU tests hold
lora_qk_rope, lora_kv_append, lora_attn_decode_window and lora_attn_chunk to. Nothing here is taken from the kernels.

The bound on a rotated value y = x0 cos a - x1 sin a (x0, x1 after the norm), computed in fp32:
  * the angle: the integer's conversion to fp32, the constant 2 pi 2^-32 and the product, each within 2^-24 of at most
    pi: 3 pi 2^-24; sine and cosine of the special-function unit: within 2^-21.19 (the documented bound of __cosf in
    [-pi, pi]); together under 2^-19;
  * the norm: at most 12 additions of squares in a chain (2^-24 each, halved by the root), mean, root and two products
    of 2 units each: under 2^-20; the two products and the difference: 2 * 2^-24;
  so |dy| <= 2^-18 (|x0| + |x1|) in fp32, and rounding to BF16 adds at most 2^-8 |y|.
"""
from __future__ import annotations

import torch

import attn_refs as R

F32 = 2.0 ** -18
EVERY = 0x7fffffff


def turned(x, positions, freqs, axis, rot, inter, norm=None, eps=0.0):
    """Rows x [n, heads, d] float64, normed by `norm` [d] and rotated; positions [axes, n] integers. Returns the result
    and the sum |x0| + |x1| that its bound goes by."""
    n, heads, d = x.shape
    if norm is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * norm.double()
    y, mag = x.clone(), x.abs()
    for j in range(rot // 2):
        u, v = (2 * j, 2 * j + 1) if inter else (j, j + rot // 2)
        # whole turns taken off in exact integer arithmetic would need more than 64 bits: positions here keep
        # position * freq within what float64 resolves to 2^-30
        a = (positions[axis[j]].double() * freqs[j])[:, None]
        y[..., u] = x[..., u] * torch.cos(a) - x[..., v] * torch.sin(a)
        y[..., v] = x[..., v] * torch.cos(a) + x[..., u] * torch.sin(a)
        mag[..., u] = mag[..., v] = x[..., u].abs() + x[..., v].abs()
    return y, mag


def seen(n, total, window, sinks, device="cuda"):
    """[n, total] bool: what the last n of `total` tokens see."""
    p = torch.arange(total - n, total, device=device)[:, None]
    t = torch.arange(total, device=device)
    return (t <= p) & ((t > p - window) | (t < sinks))


def chunk_want(q, kval, vval, table, cu, lens, page, scale, q_heads, window=EVERY, sinks=0, rounded=0.0):
    """(out [total_q, q_heads, D], lse, bound, covered rows) in 64 bits; pages outside the cache are left out. rounded:
    K's and V's elements may be off by so much of themselves (lora_attn_chunk holds codes times scales in 11 bits): a score
    by dz = rounded * scale * sum |q k|, so every weight over their sum by a factor within e^(+-2 dz); V by its part."""
    kv, D = kval.shape[1], kval.shape[3]
    G = q_heads // kv
    dev = q.device
    out = torch.zeros(q.shape[0], q_heads, D, dtype=torch.float64, device=dev)
    lse = torch.full((q.shape[0], q_heads), -torch.inf, dtype=torch.float64, device=dev)
    bound = torch.zeros_like(out)
    covered = torch.zeros(q.shape[0], dtype=torch.bool, device=dev)
    for b in range(len(cu) - 1):
        n, m = cu[b + 1] - cu[b], max(0, min(lens[b], table.shape[1] * page))
        if n <= 0 or cu[b] < 0 or cu[b + 1] > q.shape[0]:
            continue
        rows = slice(cu[b], cu[b + 1])
        covered[rows] = True
        t = torch.arange(m, device=dev)
        pg = table[b].long()[t // page]
        ok = (pg >= 0) & (pg < kval.shape[0])
        vis = seen(n, m, window, sinks, dev)[:, ok]
        pg, sl = pg[ok], (t % page)[ok]
        for h in range(q_heads):
            o, l, e = R.attend(q[rows].double().view(n, q_heads, D)[:, h], kval[pg, h // G, sl], vval[pg, h // G, sl], scale, vis)
            if rounded and vis.any():
                a, k, v = q[rows].double().view(n, q_heads, D)[:, h], kval[pg, h // G, sl], vval[pg, h // G, sl]
                used = vis.any(0)
                dz = rounded * torch.where(vis[:, used], scale * (a.abs() @ k[used].abs().T), 0.0).amax(1, keepdim=True)
                z = torch.where(vis[:, used], scale * (a @ k[used].T), -torch.inf)
                e = e + (torch.expm1(2 * dz) + rounded) * (torch.softmax(z, 1).nan_to_num(0) @ v[used].abs())
            out[rows, h], lse[rows, h], bound[rows, h] = o, l, e
    return out, lse, bound, covered
