"""Attention of one new token per sequence over the paged cache, against the 64-bit form within
the bound derived in tests/attn_refs.py (-m gpu)."""
from __future__ import annotations

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
    L.lora_read_device_status(clear=True)
    yield
    assert L.lora_read_device_status(clear=True) == 0


def case(seed, lens, kv, G, d, page, fmt, layout="hnd", spread=1.0, extra=3, kspread=None):
    g = A.gen(seed)
    num = sum(-(-n // page) for n in lens) + extra
    k, v = A.randn(g, num, kv, page, d, spread=kspread or 1.0), A.randn(g, num, kv, page, d)
    cache, kval, vval = A.cache_from_values(k, v, fmt, layout)
    table = A.block_table(g, lens, page, num)
    q = A.randn(g, len(lens), kv * G * d, spread=spread)
    return cache, kval, vval, table, q


def compare(cache, kval, vval, table, q, lens, q_heads, scale, page, **kw):
    lse = torch.full((q.shape[0], q_heads), 5.0, device="cuda")
    out = A.run_decode(q, cache, table, A.int32(lens), q_heads, scale, lse=lse, **kw)
    want, wl, bound = A.decode_want(q, kval, vval, table, lens, page, scale, q_heads)
    R.check(out.view(want.shape), want, bound, "out")
    mag = scale * q.double().abs().amax() * kval.abs().nan_to_num(0, 0, 0).amax() * kval.shape[3]
    R.check_lse(lse, wl, mag, "lse")
    return out


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kv,G", [(1, 1), (2, 2), (3, 3), (2, 5), (4, 8), (1, 16), (2, 17), (1, 40)])
def test_heads(fmt, d, kv, G):
    lens = [1, 0, 17, 130, 333]
    c = case(kv * 100 + G, lens, kv, G, d, 16, fmt)
    compare(*c, lens, kv * G, d ** -0.5, 16)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("page", [1, 3, 16, 20, 64, 128, 1000])
def test_page_sizes_and_lengths_around_them(fmt, page):
    lens = sorted({1, 2, max(1, page - 1), page, page + 1, 2 * page, 2 * page + 1, 63, 64, 65, 257})
    c = case(page, lens, 2, 4, 128, page, fmt)
    compare(*c, lens, 8, 0.1, page)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("layout", ["nhd", "kv"])
@pytest.mark.parametrize("d", [64, 128])
def test_layouts_and_strides(fmt, layout, d):
    """Other page layouts; q as a part of wider rows, out as columns of a wider buffer that stay
    otherwise untouched; a table with a stride of its own."""
    lens, kv, G, page = [5, 77, 200], 2, 4, 16
    cache, kval, vval, table, q = case(7, lens, kv, G, d, page, fmt, layout)
    H = kv * G
    rows = torch.full((3, 16 + H * d + 2 * kv * d), 9.0, dtype=torch.bfloat16, device="cuda")
    rows[:, 16:16 + H * d] = q
    wide = torch.full((3, H * d + 40), 3.0, dtype=torch.bfloat16, device="cuda")
    wt = torch.full((3, table.shape[1] + 5), 77777, dtype=torch.int32, device="cuda")
    wt[:, :table.shape[1]] = table
    A.run_decode(rows[:, 16:16 + H * d], cache, wt, A.int32(lens), H, d ** -0.5, out=wide[:, 24:24 + H * d],
                 max_pages=table.shape[1])
    want, _, bound = A.decode_want(q, kval, vval, table, lens, page, d ** -0.5, H)
    R.check(wide[:, 24:24 + H * d].reshape(want.shape), want, bound)
    assert (wide[:, :24] == 3).all() and (wide[:, 24 + H * d:] == 3).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("batch,longest,kv,G,d", [(1, 40001, 2, 8, 128), (1, 9000, 1, 1, 64), (3, 30000, 8, 1, 64),
                                                  (70, 700, 4, 4, 128), (300, 90, 2, 8, 64), (17, 5000, 8, 5, 128)])
def test_long_and_many(fmt, batch, longest, kv, G, d):
    """Lengths that spread over many blocks and batches of many short sequences, ragged."""
    r = torch.Generator().manual_seed(batch)
    lens = (torch.rand(batch, generator=r) * longest).int().tolist()
    lens[batch // 2] = longest
    c = case(batch, lens, kv, G, d, 32, fmt)
    compare(*c, lens, kv * G, d ** -0.5, 32)


@pytest.mark.parametrize("fmt", FMTS)
def test_pages_outside_the_cache_are_left_out(fmt):
    lens, page = [100, 64, 40, 16], 16
    cache, kval, vval, table, q = case(11, lens, 2, 4, 128, page, fmt)
    table[0, 2], table[0, 6] = -5, kval.shape[0]          # in the middle and at the end
    table[1, :4] = -1                                     # a sequence without any page
    table[3, 0] = 2 ** 31 - 1
    out = compare(cache, kval, vval, table, q, lens, 8, 0.09, page)
    assert (out[1] == 0).all() and (out[3] == 0).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("page", [16, 24, 64])
def test_unused_slots_may_hold_anything(fmt, page):
    """NaN and infinities in the slots past a sequence's length and in pages of nobody change nothing."""
    lens = [1, page - 3, page + 5, 3 * page - 1, 200]
    g = A.gen(13)
    num = sum(-(-n // page) for n in lens) + 2
    k, v = A.randn(g, num, 2, page, 128), A.randn(g, num, 2, page, 128)
    table = A.block_table(g, lens, page, num)
    cache, kval, vval = A.cache_from_values(k, v, fmt)
    used = torch.zeros(num, page, dtype=torch.bool, device="cuda")
    for b, n in enumerate(lens):
        t = torch.arange(n, device="cuda")
        used[table[b].long()[t // page], t % page] = True
    q = A.randn(g, len(lens), 8 * 128)
    kp, vp, ks, vs = cache.tensors
    for i, p in enumerate((kp, vp)):
        raw = p.view(torch.int16) if fmt == "bf16" else p.view(torch.uint8)
        bad = {"bf16": [0x7FC0, 0x7F80], "e4m3": [0x7F, 0xFF], "int8": [0x80, 0x7F]}[fmt]
        raw.transpose(1, 2)[~used] = bad[i]
    for s in (ks, vs):
        if s is not None:
            s.transpose(1, 2)[~used] = float("nan")
    compare(cache, kval, vval, table, q, lens, 8, 0.09, page)


@pytest.mark.parametrize("fmt", FMTS)
def test_extreme_scores_and_values(fmt):
    """Scores that differ by thousands (one key takes all), values and scales over many orders of
    magnitude from token to token."""
    lens, page, d = [300, 77], 16, 128
    c = case(17, lens, 2, 4, d, page, fmt, spread=30.0, kspread=30.0)
    compare(*c, lens, 8, 0.3, page)
    g = A.gen(19)
    num = 30
    k = A.randn(g, num, 2, page, d)
    size = torch.exp2(torch.randint(-60, 60, (num, 2, page, 1), generator=g, device="cuda").float())
    v = (A.randn(g, num, 2, page, d).float() * size).bfloat16()
    v[3] = 0
    cache, kval, vval = A.cache_from_values(k, v, fmt)
    table = A.block_table(g, lens, page, num)
    q = A.randn(g, 2, 8 * d, spread=4.0)
    compare(cache, kval, vval, table, q, lens, 8, 1.0, page)


def test_a_token_that_is_not_finite():
    """A row of the cache that is not finite reaches the outputs of its own sequence and head alone."""
    lens, page, d = [50, 60], 16, 64
    for fmt in FMTS:
        cache, kval, vval, table, q = case(23, lens, 2, 2, d, page, fmt)
        pg, sl = int(table[0, 1]), 3
        kp, vp, ks, vs = cache.tensors
        if fmt == "bf16":
            vp[pg, 1, sl, 5] = float("nan")
        else:
            vs[pg, 1, sl] = float("nan")
        out = A.run_decode(q, cache, table, A.int32(lens), 4, 0.1).view(2, 4, d)
        want, _, bound = A.decode_want(q, kval, vval, table, lens, page, 0.1, 4)
        R.check(out[1], want[1], bound[1])
        R.check(out[0, :2], want[0, :2], bound[0, :2])
        hurt = torch.isnan(out[0, 2:])
        assert hurt[:, 5].all() if fmt == "bf16" else hurt.all()


def test_nan_codes_in_a_foreign_cache():
    """E4M3 NaN codes, which lora_kv_write never makes, as the formula has them: one in K makes the rows
    that read its token NaN, one in V their results of that dimension; all others stay."""
    lens, page, d = [50, 60], 16, 128
    for which in (0, 1):
        for byte in (0x7F, 0xFF):
            cache, kval, vval, table, q = case(25, lens, 2, 2, d, page, "e4m3")
            cache.tensors[which].view(torch.uint8)[int(table[0, 2]), 1, 9, 77] = byte
            out = A.run_decode(q, cache, table, A.int32(lens), 4, 0.1).view(2, 4, d)
            want, _, bound = A.decode_want(q, kval, vval, table, lens, page, 0.1, 4)
            R.check(out[1], want[1], bound[1])
            R.check(out[0, :2], want[0, :2], bound[0, :2])
            hurt = torch.isnan(out[0, 2:])
            if which == 0:
                assert hurt.all()
            else:
                rest = [i for i in range(d) if i != 77]
                assert hurt[:, 77].all()
                R.check(out[0, 2:, rest], want[0, 2:, rest], bound[0, 2:, rest])


def test_lengths_are_clamped():
    """Negative lengths are empty, lengths past the table end with the table."""
    page, d = 16, 64
    cache, kval, vval, table, q = case(29, [32, 32, 32], 1, 2, d, page, "bf16")
    out = A.run_decode(q, cache, table, A.int32([-7, 1000, 2 ** 31 - 1]), 2, 0.2)
    want, _, bound = A.decode_want(q, kval, vval, table, [-7, 1000, 2 ** 31 - 1], page, 0.2, 2)
    R.check(out.view(want.shape), want, bound)
    assert (out[0] == 0).all()
    empty = A.run_decode(q, cache, table[:, :0], A.int32([4, 5, 6]), 2, 0.2)
    assert (empty == 0).all()


@pytest.mark.parametrize("fmt", FMTS)
def test_offsets_past_32_bits(fmt):
    d, page, kv, G = 128, 64, 2, 4
    size = 2 if fmt == "bf16" else 1
    far = (3 << 30) // size
    buf = torch.zeros(2 * far * size + 2 * kv * page * d * size, dtype=torch.uint8, device="cuda").view(R.DTYPE[fmt])
    shape, stride = (3, kv, page, d), (far, page * d, d, 1)
    views = [torch.as_strided(buf, shape, stride, o) for o in (0, kv * page * d)]
    lens = [150]
    cache, kval, vval, table, q = case(31, lens, kv, G, d, page, fmt, extra=0)
    for to, x in zip(views, cache.tensors):
        to.copy_(x)
    wide = L.KvCache(*views, *cache.tensors[2:])
    compare(wide, kval, vval, table, q, lens, kv * G, 0.1, page)


def test_same_bits_every_time_and_workspace_reuse():
    """Repeated calls give the same bits; one workspace serves calls of other shapes in between."""
    ws = A.workspace()
    a = case(37, [5000, 40, 0, 900], 4, 8, 128, 16, "bf16")
    b = case(41, [300] * 40, 2, 3, 64, 20, "int8")
    la, lb = A.int32([5000, 40, 0, 900]), A.int32([300] * 40)
    first = [A.run_decode(a[4], a[0], a[3], la, 32, 0.09, ws=ws), A.run_decode(b[4], b[0], b[3], lb, 6, 0.09, ws=ws)]
    for _ in range(20):
        assert torch.equal(A.run_decode(a[4], a[0], a[3], la, 32, 0.09, ws=ws), first[0])
        assert torch.equal(A.run_decode(b[4], b[0], b[3], lb, 6, 0.09, ws=ws), first[1])


def test_graph_replay_with_new_lengths_and_stream():
    lens = [40, 700, 3]
    cache, kval, vval, table, q = case(43, [1024, 1024, 1024], 2, 4, 128, 16, "e4m3")
    lt, ws = A.int32(lens), A.workspace()
    out = torch.zeros(3, 8 * 128, dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        A.run_decode(q, cache, table, lt, 8, 0.09, ws=ws, out=out, stream=s)
    for new in (lens, [1024, 0, 511], [1, 1, 1]):
        lt.copy_(A.int32(new))
        graph.replay()
        torch.cuda.synchronize()
        want, _, bound = A.decode_want(q, kval, vval, table, new, 16, 0.09, 8)
        R.check(out.view(want.shape), want, bound)
