"""The step's calls together, as a serving program runs them: rows normed, rotated and appended to a paged cache, chunks and
single tokens attending over it, plain and in the example layer (-m gpu)."""
from __future__ import annotations

import pytest
import torch

import attn_refs as R
import attn_util as A
import step_refs as S
from gather_lora_gb300 import lib as L
from gather_lora_gb300 import serve_step
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    require_gpu()
    L.lora_read_device_status(clear=True)
    yield
    assert L.lora_read_device_status(clear=True) == 0


@pytest.mark.parametrize("window,sinks", [(S.EVERY, 0), (24, 2)])
@pytest.mark.parametrize("kv,d,norms", [(2, 64, True), (1, 128, False)])
def test_layer_against_64_bits(kv, d, norms, window, sinks):
    """Prompts, a further chunk and single tokens with positions, norms and a window, BF16 cache. A rounding is off by at most
    2^-8 of its value, and evenly spread ones by half of that or less in the root mean square. Query and key take 4 each
    (projection, two in the fold, rotation): scores of order 1, sums of d products, move by at most sqrt(8) 2^-9 < 1.5 * 2^-8
    in the root mean square, and the result, a mean of V by weights e^score, by as much of itself. The value's 3, the
    attention's 2 and the output's 3 add as roots of squares, at most sqrt(8) 2^-8 < 3 * 2^-8: together under 5 * 2^-8, and 8 * 2^-8
    leaves room for a few rows whose weight is on one token."""
    rope = L.Rope(d)
    lay = serve_step.AttentionLayer(hidden=256, q_heads=4, kv_heads=kv, head_dim=d, cache="bf16", pages=60, seed=3, rotary=rope, norms=norms,
                                    window=None if window == S.EVERY else window, sinks=sinks)
    g = torch.Generator(device="cuda").manual_seed(4)
    counts, more, steps, adapters = [1, 33, 50], [17, 0, 30], 3, [1, -1, 3]
    rows = [torch.randn(n + m + steps, 256, generator=g, device="cuda").bfloat16() for n, m in zip(counts, more)]
    slots = lambda c: torch.cat([torch.full((n,), a, dtype=torch.int32, device="cuda") for n, a in zip(c, adapters)])
    got = [[p] for p in lay.prefill(torch.cat([r[:n] for r, n in zip(rows, counts)]), [0, 1, 2], counts, slots(counts)).split(counts)]
    y = lay.prefill(torch.cat([r[n:n + m] for r, n, m in zip(rows, counts, more)]), [0, 1, 2], more, slots(more)).split(more)
    for k in range(3):
        got[k].append(y[k])
    for k in range(steps):
        y = lay.decode(torch.stack([r[n + m + k] for r, n, m in zip(rows, counts, more)]), [0, 1, 2], slots([1, 1, 1]))
        for s in range(3):
            got[s].append(y[s:s + 1])

    def project(x, w, names, s):
        out, col = x @ w.double().T, 0
        for name in names:
            a, b = (t.double() for t in lay.adapters[name][:2])
            if adapters[s] >= 0:
                out[:, col:col + b.shape[1]] += 2.0 * (x @ a[adapters[s]].T) @ b[adapters[s]].T
            col += b.shape[1]
        return out
    freqs = [10000.0 ** (-2.0 * j / d) for j in range(d // 2)]
    for s, r in enumerate(rows):
        n, G = r.shape[0], 4 // kv
        q, k, v = project(r.double(), lay.w_qkv, "qkv", s).split(lay.widths, 1)
        at = torch.arange(n, device="cuda")[None]
        q, k = (S.turned(t.view(n, -1, d), at, freqs, [0] * (d // 2), d, False, w, 1e-6)[0] for t, w in zip((q, k), lay.norms))
        k, v = k.repeat_interleave(G, 1), v.view(n, kv, d).repeat_interleave(G, 1)
        z = torch.einsum("ihd,jhd->hij", q, k) * d ** -0.5
        z = z.masked_fill(~S.seen(n, n, window, sinks), -torch.inf)
        a = torch.einsum("hij,jhd->ihd", torch.softmax(z, -1), v).reshape(n, 4 * d)
        want = project(a, lay.w_o, "o", s)
        have = torch.cat(got[s]).double()
        off = ((have - want).norm() / want.norm()).item()
        assert off < 8 * 2.0 ** -8, (s, off)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "int8"])
@pytest.mark.parametrize("window,sinks", [(S.EVERY, 0), (50, 3)])
def test_chunk_and_single_token_forms_agree(fmt, window, sinks):
    """Appended rows read by both attentions, with one row a sequence: each within its own bound of the same 64-bit form, which
    reads the cache back."""
    kv, G, d, page, lens = 2, 4, 128, 16, [1, 90, 257, 40]
    g = A.gen(11)
    num = sum(-(-n // page) for n in lens)
    cache, _, _ = A.cache_from_values(torch.zeros(num, kv, page, d, device="cuda"), torch.zeros(num, kv, page, d, device="cuda"), fmt, "hnd")
    table = A.block_table(g, lens, page, num)
    total = sum(lens)
    at = torch.cat([torch.arange(n) for n in lens]).int().cuda()
    slots = torch.cat([table[b].long()[torch.arange(n, device="cuda") // page] * page + torch.arange(n, device="cuda") % page for b, n in enumerate(lens)])
    q, k, v = (A.randn(g, total, h * d) for h in (kv * G, kv, kv))
    L.lora_kv_append(q, q.stride(0), q, q.stride(0), kv * G, k, k.stride(0), v, v.stride(0), slots, total, cache, L.Rope(d), at, total)
    last = torch.tensor(lens).cumsum(0) - 1
    q = q[last.cuda()].contiguous()
    back = torch.empty(2, total, kv * d, dtype=torch.bfloat16, device="cuda")
    L.lora_kv_read(back[0], kv * d, back[1], kv * d, slots, total, cache)
    kval, vval = torch.zeros(2, num, kv, page, d, dtype=torch.float64, device="cuda")
    for pool, rows, scales in ((kval, 0, cache.tensors[2]), (vval, 1, cache.tensors[3])):
        codes = cache.tensors[rows].double()
        pool[slots // page, :, slots % page] = (codes * scales.double()[..., None] if fmt != "bf16" else codes)[slots // page, :, slots % page]
        read = pool[slots // page, :, slots % page].reshape(total, kv * d)
        assert ((back[rows].double() - read).abs() <= read.abs() * 2.0 ** -8).all()
    lengths, scale, h = A.int32(lens), d ** -0.5, kv * G
    one, chunk = torch.empty_like(q), torch.empty_like(q)
    ws, cws = A.workspace(), torch.empty(L.CHUNK_WORKSPACE, dtype=torch.uint8, device="cuda")
    cu = list(range(len(lens) + 1))
    L.lora_attn_decode_window(q, h * d, one, h * d, len(lens), h, scale, cache, table, table.stride(0), table.shape[1], lengths, window, sinks, ws, ws.numel())
    L.lora_attn_chunk(q, h * d, chunk, h * d, A.int32(cu), len(lens), len(lens), h, scale, cache, table, table.stride(0), table.shape[1], lengths,
                      window, sinks, cws, cws.numel())
    for out, rounded in ((one, 0.0), (chunk, 0.0 if fmt == "bf16" else 1.01 * 2.0 ** -12)):
        want, _, bound, _ = S.chunk_want(q, kval, vval, table, cu, lens, page, scale, h, window, sinks, rounded)
        # (beside an 8-bit cache the chunk's weights have a floor of 2^-32 of a row's largest a token)
        R.check(out.view(want.shape), want, bound + (2.0 ** -32 * max(lens) * vval.abs().amax() if rounded else 0), (fmt, window))


@pytest.mark.parametrize("fmt", ["bf16", "int8"])
def test_offsets_past_32_bits(fmt):
    """Pages 3 GiB apart: rows appended and read by both attentions."""
    kv, G, page, d, lens, size = 2, 2, 64, 64, [180], 2 if fmt == "bf16" else 1
    far = (3 << 30) // size
    pages = []
    for _ in range(2):
        buf = torch.zeros(2 * far * size + kv * page * d * size, dtype=torch.uint8, device="cuda").view(R.DTYPE[fmt])
        pages.append(buf.as_strided((3, kv, page, d), (far, page * d, d, 1)))
    near, _, _ = A.cache_from_values(torch.zeros(3, kv, page, d, device="cuda"), torch.zeros(3, kv, page, d, device="cuda"), fmt)
    scales = [None if t is None else torch.zeros_like(t) for t in near.tensors[2:]]
    g = A.gen(12)
    table, n, h = A.int32([[2, 0, 1]]), lens[0], kv * G
    at = torch.arange(n, device="cuda").int()
    slots = table[0].long()[at.long() // page] * page + at.long() % page
    q, k, v = (A.randn(g, n, m * d) for m in (h, kv, kv))
    ws, cws = A.workspace(), torch.empty(L.CHUNK_WORKSPACE, dtype=torch.uint8, device="cuda")
    results = []
    for cache in (near, L.KvCache(*pages, *scales)):
        turned, one, chunk = torch.empty_like(q), torch.empty_like(q[:1]), torch.empty_like(q)
        L.lora_kv_append(q, q.stride(0), turned, q.stride(0), h, k, k.stride(0), v, v.stride(0), slots, n, cache, L.Rope(d), at, n)
        args = cache, table, 3, 3, A.int32(lens), 100, 4
        L.lora_attn_decode_window(turned[n - 1:], h * d, one, h * d, 1, h, 0.125, *args, ws, ws.numel())
        L.lora_attn_chunk(turned, h * d, chunk, h * d, A.int32([0, n]), 1, n, h, 0.125, *args, cws, cws.numel())
        results.append((cache.tensors[0].contiguous(), cache.tensors[1].contiguous(), one, chunk))
    for a, b in zip(*results):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert results[0][3].abs().sum() > 0
