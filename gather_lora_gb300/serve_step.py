"""One attention layer of a multi-LoRA serving step, end to end through the library's calls.

    x -> [Q|K|V] = x W^T            (torch.matmul: the base projection)
      -> lora_bgmv on the Q, K and V columns in place   (per-request adapters)
      -> lora_kv_write              (the new K and V rows into their cache pages)
      -> lora_attn_prefill / lora_attn_decode
      -> y = a Wo^T, lora_bgmv on y

`AttentionLayer` holds the weights, adapters, paged cache and workspace that a serving program keeps;
`prefill` takes prompts, or further chunks of prompts whose first part is cached (read back with
lora_kv_read), `decode` one new token per sequence. Pages come from a plain free list.

    python -m gather_lora_gb300.serve_step        # a small run on the current GPU, checked against itself

There is no position encoding, normalisation or MLP here: the layer shows how the calls fit together.
"""
from __future__ import annotations

import torch

from . import lib as L


class AttentionLayer:
    def __init__(self, hidden=512, q_heads=8, kv_heads=2, head_dim=64, max_loras=4, rank=16, pages=64, page_size=16,
                 cache="e4m3", device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        self.hidden, self.hq, self.hkv, self.d, self.rank, self.max_loras = hidden, q_heads, kv_heads, head_dim, rank, max_loras
        self.page_size, self.device = page_size, torch.device(device)
        self.widths = (q_heads * head_dim, kv_heads * head_dim, kv_heads * head_dim)

        def weight(n, k, std=None):
            return (torch.randn(n, k, generator=g, device=device) * (std or k ** -0.5)).bfloat16()
        self.w_qkv, self.w_o = weight(sum(self.widths), hidden), weight(hidden, self.widths[0])
        # adapters of the four projections: pools, and the tables of device pointers that the folds take
        self.adapters = {}
        for name, k_in, n_out in (("q", hidden, self.widths[0]), ("k", hidden, self.widths[1]), ("v", hidden, self.widths[2]),
                                  ("o", self.widths[0], hidden)):
            a = torch.stack([weight(rank, k_in) for _ in range(max_loras)])
            b = torch.stack([weight(n_out, rank, 0.05) for _ in range(max_loras)])
            tables = [torch.tensor([t[s].data_ptr() for s in range(max_loras)], device=device) for t in (a, b)]
            self.adapters[name] = (a, b, *tables)
        self.lora_scale = torch.full((max_loras,), 2.0, device=device)
        # the cache
        dtype = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}[cache]
        shape = (pages, kv_heads, page_size, head_dim)
        pools = [torch.zeros(shape, dtype=dtype, device=device) for _ in range(2)]
        scales = [torch.zeros(shape[:3], device=device) for _ in range(2)] if cache != "bf16" else [None, None]
        self.cache = L.KvCache(*pools, *scales)
        self.free = list(range(pages))
        self.tables = {}                     # sequence -> its pages
        self.lengths = {}                    # sequence -> cached tokens
        self.workspace = torch.zeros(L.ATTN_WORKSPACE, dtype=torch.uint8, device=device)

    def _fold(self, name, x, out, column, seq_slot):
        """The adapters of projection `name` folded into out[:, column : column + n_out], in place."""
        a, b, a_table, b_table = self.adapters[name]
        L.lora_bgmv(x, x.stride(0), out.data_ptr() + 2 * column, out.stride(0), seq_slot, x.shape[0], a_table, b_table,
                    self.lora_scale, self.max_loras, self.rank, a.shape[2], b.shape[1])

    def _qkv(self, x, seq_slot):
        qkv = x @ self.w_qkv.T
        column = 0
        for name, width in zip("qkv", self.widths):
            self._fold(name, x, qkv, column, seq_slot)
            column += width
        return qkv

    def _out(self, a, seq_slot):
        y = a @ self.w_o.T
        self._fold("o", a, y, 0, seq_slot)
        return y

    def _check(self, x, seqs, counts, seq_slot):
        """Refuse a call before any of it changes the layer: rows that do not fit, a sequence twice, too few free pages."""
        if (x.dim() != 2 or x.shape != (sum(counts), self.hidden) or x.stride(1) != 1 or len(seqs) != len(counts) or
                min(counts, default=0) < 0):
            raise ValueError(f"rows {tuple(x.shape)} for {len(seqs)} sequences with {list(counts)} rows of {self.hidden}")
        if seq_slot.shape != (x.shape[0],) or seq_slot.dtype != torch.int32:
            raise ValueError(f"seq_slot is int32 [{x.shape[0]}]: got {seq_slot.dtype} {tuple(seq_slot.shape)}")
        if len(set(seqs)) != len(seqs):
            raise ValueError(f"a sequence is there twice: {list(seqs)}")
        need = sum(max(0, -(-(self.lengths.get(s, 0) + n) // self.page_size) - len(self.tables.get(s, [])))
                   for s, n in zip(seqs, counts))
        if need > len(self.free):
            raise RuntimeError(f"{need} pages are needed, {len(self.free)} are free: release a sequence first")

    def _slots(self, seq, first, n):
        """Cache slots of tokens first .. first + n of a sequence, pages taken as they are needed."""
        pages = self.tables.setdefault(seq, [])
        while len(pages) * self.page_size < first + n:
            pages.append(self.free.pop())
        t = torch.arange(first, first + n)
        return torch.tensor(pages, dtype=torch.int64)[t // self.page_size] * self.page_size + t % self.page_size

    def _write(self, qkv, slots):
        q, k, _ = self.widths
        L.lora_kv_write(qkv.data_ptr() + 2 * q, qkv.stride(0), qkv.data_ptr() + 2 * (q + k), qkv.stride(0), slots,
                        qkv.shape[0], self.cache)

    def prefill(self, x, seqs, counts, seq_slot):
        """Rows x [sum(counts), hidden] of the sequences `seqs`, each after what of it is cached already."""
        self._check(x, seqs, counts, seq_slot)
        before = [self.lengths.get(s, 0) for s in seqs]
        slots = torch.cat([self._slots(s, b, n) for s, b, n in zip(seqs, before, counts)]).to(self.device)
        qkv = self._qkv(x, seq_slot)
        self._write(qkv, slots)
        for s, b, n in zip(seqs, before, counts):
            self.lengths[s] = b + n
        q, kv = self.widths[0], self.widths[1]
        cu_q, cu_k = ([0], [0])
        for b, n in zip(before, counts):
            cu_q.append(cu_q[-1] + n)
            cu_k.append(cu_k[-1] + b + n)
        if any(before):       # chunks: keys and values of the cached parts and the new rows, read back into rows of their own
            every = torch.cat([self._slots(s, 0, b + n) for s, b, n in zip(seqs, before, counts)]).to(self.device)
            k, v = (torch.empty(every.numel(), kv, dtype=torch.bfloat16, device=self.device) for _ in range(2))
            L.lora_kv_read(k, kv, v, kv, every, every.numel(), self.cache)
        else:
            k, v = qkv[:, q:q + kv], qkv[:, q + kv:]
        a = torch.empty(x.shape[0], q, dtype=torch.bfloat16, device=self.device)
        starts = [torch.tensor(c, dtype=torch.int32, device=self.device) for c in (cu_q, cu_k)]
        L.lora_attn_prefill(qkv, qkv.stride(0), k, k.stride(0), v, v.stride(0), a, q, *starts, len(seqs), x.shape[0],
                            k.shape[0], self.hq, self.hkv, self.d, self.d ** -0.5)
        return self._out(a, seq_slot)

    def decode(self, x, seqs, seq_slot):
        """One new token per sequence: x [len(seqs), hidden]."""
        self._check(x, seqs, [1] * len(seqs), seq_slot)
        slots = torch.cat([self._slots(s, self.lengths.get(s, 0), 1) for s in seqs]).to(self.device)
        qkv = self._qkv(x, seq_slot)
        self._write(qkv, slots)
        for s in seqs:
            self.lengths[s] = self.lengths.get(s, 0) + 1
        width = max(len(self.tables[s]) for s in seqs)
        table = torch.tensor([self.tables[s] + [-1] * (width - len(self.tables[s])) for s in seqs], dtype=torch.int32,
                             device=self.device)
        lens = torch.tensor([self.lengths[s] for s in seqs], dtype=torch.int32, device=self.device)
        q = self.widths[0]
        a = torch.empty(x.shape[0], q, dtype=torch.bfloat16, device=self.device)
        L.lora_attn_decode(qkv, qkv.stride(0), a, q, len(seqs), self.hq, self.d ** -0.5, self.cache, table, width, width, lens,
                           self.workspace, self.workspace.numel())
        return self._out(a, seq_slot)

    def release(self, seq):
        self.free.extend(self.tables.pop(seq, []))
        self.lengths.pop(seq, None)


def main() -> None:
    """Three requests with different adapters: prompts, a second chunk for one, then decode steps; the
    same rows through one prefill call on a fresh layer must agree (the cache's rounding apart)."""
    counts, extra, steps, hidden = [37, 5, 70], 20, 3, 512
    g = torch.Generator(device="cuda").manual_seed(1)
    for cache, most in (("bf16", 0.02), ("int8", 0.03), ("e4m3", 0.1)):
        layer, whole = (AttentionLayer(hidden, cache=c) for c in (cache, "bf16"))
        adapter = [0, -1, 2]
        rows = [torch.randn(n + (extra if s == 1 else 0) + steps, hidden, generator=g, device="cuda").bfloat16()
                for s, n in enumerate(counts)]
        slot = [torch.full((r.shape[0],), adapter[s], dtype=torch.int32, device="cuda") for s, r in enumerate(rows)]
        got = [[] for _ in rows]
        y = layer.prefill(torch.cat([r[:n] for r, n in zip(rows, counts)]), [0, 1, 2], counts,
                          torch.cat([t[:n] for t, n in zip(slot, counts)]))
        for s, part in enumerate(y.split(counts)):
            got[s].append(part)
        got[1].append(layer.prefill(rows[1][5:25], [1], [extra], slot[1][5:25]))
        for step in range(steps):
            at = [r.shape[0] - steps + step for r in rows]
            y = layer.decode(torch.stack([r[i] for r, i in zip(rows, at)]), [0, 1, 2], torch.stack([t[i] for t, i in zip(slot, at)]))
            for s in range(3):
                got[s].append(y[s:s + 1])
        want = whole.prefill(torch.cat(rows), [0, 1, 2], [r.shape[0] for r in rows], torch.cat(slot))
        have = torch.cat([torch.cat(p) for p in got])
        off = ((have.double() - want.double()).norm() / want.double().norm()).item()
        print(f"cache {cache}: {have.shape[0]} rows over prompts, a chunk and decode steps, {off:.4f} off one prefill")
        assert off < most, (cache, off)


if __name__ == "__main__":
    main()
