"""Inputs for the cache and attention tests on the GPU: pools with chosen layouts, block tables,
packed sequences, and the 64-bit results for them (tests/attn_refs.py)."""
from __future__ import annotations

import numpy as np
import torch

import attn_refs as R
from gather_lora_gb300 import lib as L

DEV = "cuda"


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def randn(g, *shape, spread=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * spread).bfloat16()


def pool(num_pages, kv, page, d, fmt, layout="hnd", fill=None):
    """(k_pages, v_pages) views [num_pages, kv, page, d] of fresh storage in the given layout:
    hnd, nhd, or kv (the K and V pages interleaved in one buffer). fill: the byte everywhere."""
    size = 2 if fmt == "bf16" else 1

    def storage(*shape):
        n = int(np.prod(shape)) * size
        t = torch.full((max(n, 1),), 0 if fill is None else fill, dtype=torch.uint8, device=DEV)
        return t[:n].view(R.DTYPE[fmt]).view(*shape)
    if layout == "hnd":
        return storage(num_pages, kv, page, d), storage(num_pages, kv, page, d)
    if layout == "nhd":
        return (storage(num_pages, page, kv, d).transpose(1, 2), storage(num_pages, page, kv, d).transpose(1, 2))
    both = storage(num_pages, 2, kv, page, d)
    return both[:, 0], both[:, 1]


def cache_from_values(k, v, fmt, layout="hnd"):
    """A cache holding the given [num_pages, kv, page, d] bf16 values (quantised by the reference in
    the 8-bit formats), with the float64 values that it stands for."""
    out = []
    pages = pool(*k.shape, fmt, layout)
    scales = []
    for x, p in zip((k, v), pages):
        if fmt == "bf16":
            p.copy_(x)
            out.append(x.double())
            continue
        code, s = R.quantise(x.float().cpu().numpy(), fmt)
        p.copy_(torch.from_numpy(code).to(DEV).float().to(R.DTYPE[fmt]))
        scales.append(torch.from_numpy(s).to(DEV))
        out.append(torch.from_numpy(code * s.astype(np.float64)[..., None]).to(DEV))
    return L.KvCache(*pages, *scales), out[0], out[1]


def workspace():
    return torch.zeros(L.ATTN_WORKSPACE, dtype=torch.uint8, device=DEV)


def block_table(g, lens, page, num_pages, width=None):
    """Disjoint random pages for each sequence; unused entries -1."""
    need = [-(-n // page) for n in lens]
    assert sum(need) <= num_pages
    order = torch.randperm(num_pages, generator=g, device=DEV).int()
    t = torch.full((len(lens), max(width or 0, max(need + [1]))), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, m in enumerate(need):
        t[b, :m] = order[at:at + m]
        at += m
    return t


def decode_want(q, kval, vval, table, lens, page, scale, q_heads):
    """(out [B, q_heads, D], lse, bound) in 64 bits; pages outside the cache are left out."""
    B, kv, D = q.shape[0], kval.shape[1], kval.shape[3]
    G = q_heads // kv
    out = torch.zeros(B, q_heads, D, dtype=torch.float64, device=DEV)
    lse = torch.full((B, q_heads), -torch.inf, dtype=torch.float64, device=DEV)
    bound = torch.zeros_like(out)
    for b, n in enumerate(lens):
        n = max(0, min(n, table.shape[1] * page))
        t = torch.arange(n, device=DEV)
        pg = table[b].long()[t // page]
        ok = (pg >= 0) & (pg < kval.shape[0])
        pg, sl = pg[ok], (t % page)[ok]
        for h in range(kv):
            rows = slice(h * G, (h + 1) * G)
            o, l, e = R.attend(q[b].double().view(q_heads, D)[rows], kval[pg, h, sl], vval[pg, h, sl], scale)
            out[b, rows], lse[b, rows], bound[b, rows] = o, l, e
    return out, lse, bound


def run_decode(q, cache, table, lens_t, q_heads, scale, ws=None, out=None, lse=None, stream=None, max_pages=None):
    d = cache.struct.head_dim
    if out is None:
        out = torch.full((q.shape[0], q_heads * d), float("nan"), dtype=torch.bfloat16, device=DEV)
    ws = workspace() if ws is None else ws
    L.lora_attn_decode(q, q.stride(0), out, out.stride(0), q.shape[0], q_heads, scale, cache, table, table.stride(0),
                       table.shape[1] if max_pages is None else max_pages, lens_t, ws, ws.numel(), lse=lse, stream=stream)
    return out


def prefill_want(q, k, v, cu_q, cu_k, q_heads, kv, scale):
    """(out [total_q, q_heads, D], lse, bound, covered rows) in 64 bits."""
    D = q.shape[1] // q_heads
    G = q_heads // kv
    out = torch.zeros(q.shape[0], q_heads, D, dtype=torch.float64, device=DEV)
    lse = torch.full((q.shape[0], q_heads), -torch.inf, dtype=torch.float64, device=DEV)
    bound = torch.zeros_like(out)
    covered = torch.zeros(q.shape[0], dtype=torch.bool, device=DEV)
    for b in range(len(cu_q) - 1):
        q0, q1, k0, k1 = cu_q[b], cu_q[b + 1], cu_k[b], cu_k[b + 1]
        n, m = q1 - q0, k1 - k0
        if n <= 0:
            continue
        covered[q0:q1] = True
        seen = torch.arange(m, device=DEV) <= torch.arange(n, device=DEV)[:, None] + (m - n)
        for h in range(q_heads):
            g = h // G
            o, l, e = R.attend(q[q0:q1, h * D:(h + 1) * D].double(), k[k0:k1, g * D:(g + 1) * D].double(),
                               v[k0:k1, g * D:(g + 1) * D].double(), scale, seen)
            out[q0:q1, h], lse[q0:q1, h], bound[q0:q1, h] = o, l, e
    return out, lse, bound, covered


def run_prefill(q, k, v, cu_q, cu_k, q_heads, kv, scale, out=None, lse=None, stream=None):
    D = q.shape[1] // q_heads
    if out is None:
        out = torch.full((q.shape[0], q_heads * D), float("nan"), dtype=torch.bfloat16, device=DEV)
    L.lora_attn_prefill(q, q.stride(0), k, k.stride(0), v, v.stride(0), out, out.stride(0), cu_q, cu_k, cu_q.numel() - 1,
                        q.shape[0], k.shape[0], q_heads, kv, D, scale, lse=lse, stream=stream)
    return out


def int32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)
