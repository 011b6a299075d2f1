"""The paged cache written and read back on the GPU (-m gpu): codes and scales are the stated
float32 formulas' bit for bit, slots outside the cache are skipped, other slots stay untouched."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import attn_refs as R
import attn_util as A
from gather_lora_gb300 import lib as L
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu
FMTS = ["bf16", "e4m3", "int8"]


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    require_gpu()


def scales(num_pages, kv, page, fmt):
    return [None, None] if fmt == "bf16" else [torch.full((num_pages, kv, page), 7.0, device="cuda") for _ in range(2)]


def as_bytes(t):
    return t.contiguous().view(torch.uint8).cpu().numpy()


def roundtrip(x, slots, pages, sc, fmt, kv, d):
    """Write rows x [n, 2 * kv * d] (K then V) and read the same slots back."""
    n = x.shape[0]
    cache = L.KvCache(*pages, *sc)
    s = x.stride(0)
    L.lora_kv_write(x, s, x.data_ptr() + kv * d * 2, s, slots, n, cache)
    out = [torch.full((n, kv * d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    L.lora_kv_read(out[0], kv * d, out[1], kv * d, slots, n, cache)
    torch.cuda.synchronize()
    return out


def expect(x, fmt):
    """(codes, scales, read back) of rows [..., d] bf16, as numpy."""
    f = x.float().cpu().numpy()
    if fmt == "bf16":
        return f, None, x.cpu()
    code, s = R.quantise(f, fmt)
    back = (code.astype(np.float32) * s[..., None]).astype(np.float32)      # exact product rounded once
    return code, s, torch.from_numpy(back).bfloat16()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("layout", ["hnd", "nhd", "kv"])
@pytest.mark.parametrize("n,kv,page", [(1, 1, 1), (3, 2, 7), (37, 4, 16), (515, 3, 64), (1000, 8, 20)])
def test_write_and_read(fmt, d, layout, n, kv, page):
    g = A.gen(n + d)
    num = -(-n // page) + 3
    pages = A.pool(num, kv, page, d, fmt, layout, fill=0x5A)
    sc = scales(num, kv, page, fmt)
    wide = A.randn(g, n, 2 * kv * d + 24, spread=3.0)     # rows wider than what is stored
    x = wide[:, 8:8 + 2 * kv * d]
    slots = torch.randperm(num * page, generator=g, device="cuda")[:n].clone()
    if n > 2:
        slots[1], slots[2] = -1, num * page                # both outside: skipped
    out = roundtrip(x, slots, pages, sc, fmt, kv, d)
    live = ((slots >= 0) & (slots < num * page)).cpu()
    pg, sl = (slots.cpu()[live] // page), (slots.cpu()[live] % page)
    for j in range(2):
        rows = x[:, j * kv * d:(j + 1) * kv * d].reshape(n, kv, d)
        code, s, back = expect(rows[live.cuda()], fmt)
        got = pages[j].cpu()[pg, :, sl] if fmt == "bf16" else pages[j].view(torch.uint8).cpu()[pg, :, sl].view(R.DTYPE[fmt])
        assert np.array_equal(got.double().numpy(), code.astype(np.float64))
        if s is not None:
            assert np.array_equal(sc[j].cpu()[pg, :, sl].numpy(), s)
        assert torch.equal(out[j].cpu()[live].view(-1, kv, d), back)
        assert (out[j].cpu()[~live].float() == 0).all()    # a slot outside reads as zeros
        # nothing else was written
        hit = torch.zeros(num, page, dtype=torch.bool)
        hit[pg, sl] = True
        rest = pages[j].view(torch.uint8) if fmt != "bf16" else pages[j].contiguous().view(torch.uint8)
        assert (rest.cpu().transpose(1, 2)[~hit] == 0x5A).all()
        if s is not None:
            assert (sc[j].cpu().transpose(1, 2)[~hit] == 7.0).all()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("d", [64, 128])
def test_rows_at_the_edges_of_the_formats(fmt, d):
    """Zero rows, tiny rows around 2^-100, huge rows, rows with one NaN or infinity, exact ties."""
    x = torch.zeros(10, 2 * d, dtype=torch.float32)
    g = torch.Generator().manual_seed(3)
    x[1] = 2.0 ** -101 * torch.rand(2 * d, generator=g)
    x[2, ::3] = 2.0 ** -100
    x[3] = 3e38 * (torch.rand(2 * d, generator=g) - 0.5)
    x[4] = torch.randn(2 * d, generator=g)
    x[4, 5] = float("nan")
    x[4, d + 7] = float("inf")
    x[5] = torch.randn(2 * d, generator=g)
    x[5, 9], x[5, d] = float("-inf"), float("nan")
    x[6] = R.QMAX[fmt]
    x[6, 1:d], x[6, d + 1:] = torch.arange(1, d) + 0.5, -(torch.arange(1, d) + 0.5)     # scale 1: ties
    x[7, 3], x[7, d + 3] = -5.0, 1e-30
    x[8] = torch.randn(2 * d, generator=g) * 1e-28
    x[9] = torch.exp(4 * torch.randn(2 * d, generator=g))
    x = x.bfloat16().cuda()
    pages, sc = A.pool(3, 1, 4, d, fmt), scales(3, 1, 4, fmt)
    slots = torch.arange(10, device="cuda")
    out = roundtrip(x, slots, pages, sc, fmt, 1, d)
    for j in range(2):
        rows = x[:, j * d:(j + 1) * d].reshape(10, 1, d)
        code, s, back = expect(rows, fmt)
        got = pages[j].view(torch.uint8).cpu().view(12, d)[:10].view(R.DTYPE[fmt]).double().numpy()
        assert np.array_equal(got, code.reshape(10, d))
        assert np.array_equal(sc[j].cpu().numpy().reshape(12)[:10], s.reshape(10), equal_nan=True)
        o = out[j].cpu().float().numpy()
        want = back.float().numpy().reshape(10, d)
        assert np.array_equal(o, want, equal_nan=True)
        assert np.isnan(o[4]).all() and np.isnan(o[5]).all() and (o[0] == 0).all() and (o[1] == 0).all()


@pytest.mark.parametrize("fmt", FMTS)
def test_slots_past_32_bits(fmt):
    """A pool whose byte offsets pass 2^32 (pages far apart), and slot numbers that do."""
    d, page, kv = 64, 16, 2
    size = 2 if fmt == "bf16" else 1
    far = (3 << 30) // size                                # elements between pages
    buf = torch.zeros(2 * far * size + 2 * kv * page * d * size, dtype=torch.uint8, device="cuda").view(R.DTYPE[fmt])
    shape, stride = (3, kv, page, d), (far, page * d, d, 1)
    pages = [torch.as_strided(buf, shape, stride, o) for o in (0, kv * page * d)]
    sc = scales(3, kv, page, fmt)
    g = A.gen(5)
    n = 3 * page
    x = A.randn(g, n, 2 * kv * d)
    slots = torch.arange(n, device="cuda")
    out = roundtrip(x, slots, pages, sc, fmt, kv, d)
    for j in range(2):
        _, _, back = expect(x[:, j * kv * d:(j + 1) * kv * d].reshape(n, kv, d), fmt)
        assert torch.equal(out[j].cpu().view(n, kv, d), back)
    # slot numbers past 2^32: pages of 2^30 tokens that all lie on the same memory (token stride 0 is refused; stride via pages)
    many = torch.tensor([1 << 33, (1 << 40) + 5, -(1 << 35)], device="cuda")
    before = as_bytes(pages[0])
    roundtrip(x[:3], many, pages, sc, fmt, kv, d)
    assert np.array_equal(before, as_bytes(pages[0]))      # outside the cache: skipped


def test_other_stream_and_graph():
    """Calls go to the given stream, and a captured write and read replay with new slots and rows."""
    d, kv, page, n = 128, 2, 8, 21
    g = A.gen(9)
    pages, sc = A.pool(6, kv, page, d, "e4m3"), scales(6, kv, page, "e4m3")
    cache = L.KvCache(*pages, *sc)
    x, slots = A.randn(g, n, 2 * kv * d), torch.randperm(48, generator=g, device="cuda")[:n].clone()
    out = [torch.zeros(n, kv * d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        L.lora_kv_write(x, 2 * kv * d, x.data_ptr() + kv * d * 2, 2 * kv * d, slots, n, cache, stream=s)
        L.lora_kv_read(out[0], kv * d, out[1], kv * d, slots, n, cache, stream=s)
    for seed in (1, 2):
        h = A.gen(seed)
        x.copy_(A.randn(h, n, 2 * kv * d))
        slots.copy_(torch.randperm(48, generator=h, device="cuda")[:n])
        graph.replay()
        torch.cuda.synchronize()
        for j in range(2):
            _, _, back = expect(x[:, j * kv * d:(j + 1) * kv * d].reshape(n, kv, d), "e4m3")
            assert torch.equal(out[j].cpu().view(n, kv, d), back)
