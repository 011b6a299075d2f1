"""Attention of chunks of new tokens over the paged cache, against the 64-bit form within the bound derived in
tests/attn_refs.py (-m gpu)."""
from __future__ import annotations

import itertools

import pytest
import torch

import attn_refs as R
import attn_util as A
import step_refs as S
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


def workspace():
    return torch.zeros(L.CHUNK_WORKSPACE, dtype=torch.uint8, device="cuda")


def starts(ns):
    return [0] + list(itertools.accumulate(ns))


def case(seed, nl, kv, G, d, page, fmt, layout="hnd", spread=1.0, extra=3):
    """nl: (new rows, cached tokens) of each sequence. q rows lie in wider rows."""
    g = A.gen(seed)
    lens = [m for _, m in nl]
    num = sum(-(-m // page) for m in lens) + extra
    k, v = A.randn(g, num, kv, page, d, spread=spread), A.randn(g, num, kv, page, d)
    cache, kval, vval = A.cache_from_values(k, v, fmt, layout)
    cu = starts([n for n, _ in nl])
    q = A.randn(g, cu[-1], kv * G * d + 24, spread=spread)[:, 8:8 + kv * G * d]
    return cache, kval, vval, A.block_table(g, lens, page, num), q, cu, lens


def run(cache, table, q, cu, lens, h, scale, window=S.EVERY, sinks=0, ws=None, out=None, lse=None, stream=None):
    d = cache.struct.head_dim
    out = torch.full((q.shape[0], h * d), float("nan"), dtype=torch.bfloat16, device="cuda") if out is None else out
    ws = workspace() if ws is None else ws
    cu, lens = (x if isinstance(x, torch.Tensor) else A.int32(x) for x in (cu, lens))
    L.lora_attn_chunk(q, q.stride(0), out, out.stride(0), cu, lens.numel(), q.shape[0], h, scale, cache, table, table.stride(0), table.shape[1],
                      lens, window, sinks, ws, ws.numel(), lse=lse, stream=stream)
    return out


# 8-bit caches: codes times scales are rounded to f16 once, half a step of 11 bits; of values 2^-29 and more below the
# group's largest, subnormal there, by 2^-40 of that largest, which the factor 1.01 covers at the sizes here.
ROUNDED = 1.01 * 2.0 ** -12


def f16_floor(vval, lens):
    """Over 8-bit caches the weights w_t s_t are kept in f16, the largest of a row between 2^7 and 2^15: one whose f16 is
    subnormal is off by at most half of 2^-24 whatever its own size, 2^-32 of the largest. With s the scale of the token
    with the largest and codes c_t, the result is off by at most 2^-32 s sum_t |c_t| <= 2^-32 (tokens) max |v|."""
    return 2.0 ** -32 * max(lens, default=0) * vval.abs().nan_to_num(0, 0, 0).amax()


def compare(cache, kval, vval, table, q, cu, lens, h, scale=0.1, window=S.EVERY, sinks=0, ws=None):
    page = cache.struct.page_size
    lse = torch.full((q.shape[0], h), 5.0, device="cuda")
    out = run(cache, table, q, cu, lens, h, scale, window, sinks, ws=ws, lse=lse)
    coded = cache.struct.format != L.KV_BF16
    want, wl, bound, covered = S.chunk_want(q, kval, vval, table, cu, lens, page, scale, h, window, sinks, rounded=ROUNDED if coded else 0.0)
    if coded:
        bound = bound + f16_floor(vval, lens)
    R.check(out.view(want.shape)[covered], want[covered], bound[covered], ("out", window, sinks))
    mag = scale * q.shape[1] / h * q.double().abs().nan_to_num(0, 0, 0).amax() * kval.abs().nan_to_num(0, 0, 0).amax() if q.shape[0] else 0
    # (the rounding of K moves a score, and so their log-sum, by ROUNDED * mag: check_lse allows 140 * 2^-24 of what it gets)
    R.check_lse(lse[covered], wl[covered], mag * (1 + (ROUNDED * 2 ** 24 / 140 if coded else 0)), "lse")
    return out


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kv,G", [(1, 1), (2, 2), (1, 3), (2, 5), (1, 7), (2, 8), (1, 16), (1, 48), (1, 130)])
def test_heads(fmt, d, kv, G):
    data = case(kv * 100 + G, [(1, 1), (33, 33), (150, 150), (0, 40), (7, 300), (1, 513), (5, 0)], kv, G, d, 16, fmt)
    compare(*data, kv * G, d ** -0.5)
    compare(*data, kv * G, d ** -0.5, 40, 3)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 255, 257, 300, 513])
def test_lengths(fmt, n):
    """One chunk of each length: alone, after a prefix, and with fewer cached tokens than rows."""
    for m in (n, n + 1, n + 130, max(0, n - 1), n // 2, n + 1000):
        for d in (64, 128):
            compare(*case(n + m, [(n, m)], 2, 4, d, 32, fmt), 8, 0.11)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d,page,layout", [(128, 1, "hnd"), (64, 8, "nhd"), (128, 20, "kv"), (64, 48, "hnd"), (128, 128, "nhd"), (64, 200, "kv"), (128, 7, "nhd")])
def test_pages_and_layouts(fmt, d, page, layout):
    data = case(page, [(40, 40), (3, 333), (130, 260), (1, 129)], 2, 3, d, page, fmt, layout)
    compare(*data, 6)
    compare(*data, 6, 0.1, 100, 10)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d,G", [(128, 4), (64, 1), (128, 16)])
def test_windows(fmt, d, G):
    """Windows and first tokens that meet, lie apart, end inside tiles, hide whole tiles of some rows and not of others."""
    data = case(d + G, [(1, 1), (200, 200), (3, 900), (300, 1100), (140, 1300), (50, 20)], 1, G, d, 16, fmt)
    for window, sinks in ((1, 0), (1, 5), (2, 1), (100, 0), (128, 128), (129, 127), (250, 300), (511, 4), (1000, 50), (1300, 0), (4, 2 ** 31 - 1), (700, 130)):
        compare(*data, G, 0.1, window, sinks)


@pytest.mark.parametrize("fmt", FMTS)
def test_packed(fmt):
    """Many sequences in one call: chunks, single tokens, empty ones and rows without tokens among them."""
    r = torch.Generator().manual_seed(4)
    nl = [(int(a) if b % 3 else 1, int(a + b * 4)) for a, b in torch.randint(0, 150, (60, 2), generator=r).tolist()]
    nl[3], nl[10], nl[20], nl[59] = (0, 50), (64, 0), (100, 30), (0, 0)
    for d, G in ((128, 4), (64, 2)):
        data = case(99 + d, nl, 2, G, d, 16, fmt)
        compare(*data, 2 * G)
        compare(*data, 2 * G, 0.1, 77, 7)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("kv,G,d,nl", [(1, 8, 128, [(1, 9000)]), (2, 4, 128, [(5, 20000), (1, 40)]), (1, 4, 64, [(2, 70000)]), (1, 8, 128, [(600, 9000)]),
                                        (4, 1, 64, [(700, 4000), (2, 16000)]), (2, 2, 128, [(1500, 1500)])])
def test_long(fmt, kv, G, d, nl):
    """Work that is shared out over many CTAs and joined: the same bits every time."""
    data = case(11, nl, kv, G, d, 64, fmt)
    ws = workspace()
    for window, sinks in ((S.EVERY, 0), (3000, 9)):
        first = compare(*data, kv * G, d ** -0.5, window, sinks, ws=ws)
        for _ in range(3):
            assert torch.equal(first, run(data[0], data[3], data[4], data[5], data[6], kv * G, d ** -0.5, window, sinks, ws=ws))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d", [64, 128])
def test_large_scores(fmt, d):
    """Scores that differ by thousands, maxima that rise along the tokens."""
    g = A.gen(6)
    page, kv, G, nl = 16, 2, 4, [(300, 300), (100, 400), (2, 2000)]
    num = sum(-(-m // page) for _, m in nl) + 1
    lens, cu = [m for _, m in nl], starts([n for n, _ in nl])
    table = A.block_table(g, lens, page, num)
    k, v = A.randn(g, num, kv, page, d, spread=12.0), A.randn(g, num, kv, page, d)
    for b, m in enumerate(lens):
        for e in range(-(-m // page)):
            k[table[b, e]] = (k[table[b, e]].float() * (0.1 + 3 * e * page / m)).bfloat16()
    cache, kval, vval = A.cache_from_values(k, v, fmt)
    compare(cache, kval, vval, table, A.randn(g, cu[-1], kv * G * d, spread=12.0), cu, lens, kv * G, 0.5)


def place(table, page, b, t):
    """(pages, slots) of tokens t of sequence b."""
    t = torch.as_tensor(t, device="cuda")
    return table[b].long()[t // page], t % page


def spoil(cache, table, page, b, t, bad):
    """Tokens t of sequence b hold `bad` in every element of K and V (8 bits: scale `bad`)."""
    pg, sl = place(table, page, b, t)
    k, v, ks, vs = cache.tensors
    for x, s in ((k, ks), (v, vs)):
        if x.dtype == torch.bfloat16:
            x[pg, :, sl] = bad
        else:
            s[pg, :, sl] = bad


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf"), torch.finfo(torch.bfloat16).min])
@pytest.mark.parametrize("d,G", [(64, 1), (128, 4)])
def test_tokens_that_are_not_seen_have_no_influence(fmt, bad, d, G):
    """Bad values in tokens that some rows see and others do not, on either side of the window: the rows that do not see
    them are as if they were not there."""
    page = 16
    nl = [(200, 260), (70, 500), (3, 130)]
    cache, kval, vval, table, q, cu, lens = case(8, nl, 1, G, d, page, fmt)
    window, sinks = 90, 5
    clean = run(cache, table, q, cu, lens, G, 0.1, window, sinks)
    every = run(cache, table, q, cu, lens, G, 0.1)
    at = {0: [100, 197, 259], 1: [300, 431, 480], 2: [2, 128]}
    for b, t in at.items():
        spoil(cache, table, page, b, t, bad)
    for w, s, want in ((window, sinks, clean), (S.EVERY, 0, every)):
        got = run(cache, table, q, cu, lens, G, 0.1, w, s)
        for b, (n, m) in enumerate(nl):
            hit = S.seen(n, m, w, s)[:, at[b]].any(1)
            rows = slice(cu[b], cu[b + 1])
            assert torch.isfinite(got[rows][~hit]).all()
            # (what they hold may be split differently from the clean call's only if it reads data: it does not)
            assert torch.equal(got[rows][~hit], want[rows][~hit]), (b, w)
            if bad != bad:
                assert torch.isnan(got[rows][hit]).all()


@pytest.mark.parametrize("d,G", [(64, 2), (128, 3)])
def test_values_that_are_not_finite_reach_those_who_see_them(d, G):
    """NaN and infinities in single elements of V (BF16): the rows that see them get them there and nowhere else, within
    and at both ends of the window; in a long context shared out over CTAs as well."""
    page, window, sinks = 16, 150, 20
    for nl in ([(200, 420), (60, 60)], [(40, 9000)]):
        cache, kval, vval, table, q, cu, lens = case(17, nl, 1, G, d, page, "bf16")
        _, v, _, _ = cache.tensors
        for b, (n, m) in enumerate(nl):
            for x, (t, e, bad) in enumerate(((m - n, 1, float("nan")), (m - 1, 5, float("inf")), (m - n // 2, 7, float("-inf")),
                                             (max(0, m - n - 100), 9, float("inf")), (m - 3, 5, float("-inf")), (4, 11, float("nan")),
                                             (m - n // 3, d - 1, float("nan")), (max(0, m - n - 149), d // 2, float("-inf")))):
                pg, sl = place(table, page, b, [t])
                v[pg, :, sl, e] = bad
                vval[pg, :, sl, e] = bad
        for w, s in ((window, sinks), (S.EVERY, 0)):
            out = run(cache, table, q, cu, lens, G, 0.1, w, s)
            want, _, bound, _ = S.chunk_want(q, kval, vval, table, cu, lens, page, 0.1, G, w, s)
            out = out.view(want.shape).double()
            assert torch.equal(torch.isnan(out), torch.isnan(want)) and torch.equal(out[torch.isinf(want)], want[torch.isinf(want)])
            fine = torch.isfinite(want)
            assert ((out - want).abs()[fine] <= bound[fine]).all()


@pytest.mark.parametrize("fmt", FMTS)
def test_bad_pages_and_unused_slots(fmt):
    """Pages outside the cache leave their tokens out; what unused slots and unused pages hold is not seen."""
    page, d, G = 16, 128, 4
    nl = [(30, 100), (90, 333), (1, 45)]
    cache, kval, vval, table, q, cu, lens = case(21, nl, 2, G, d, page, fmt)
    for x in cache.tensors[:2]:
        used = torch.zeros(x.shape[0], page, dtype=torch.bool, device="cuda")
        for b, m in enumerate(lens):
            pg, sl = place(table, page, b, list(range(m)))
            used[pg, sl] = True
        rest = (~used).nonzero()
        if fmt == "bf16":
            x[rest[:, 0], :, rest[:, 1]] = float("nan")
        else:
            x.view(torch.uint8)[rest[:, 0], :, rest[:, 1]] = 0x7F
    table = table.clone()
    table[0, 1], table[1, 5], table[1, 20], table[2, 0] = -1, 10 ** 6, kval.shape[0], -7
    for w, s in ((S.EVERY, 0), (50, 4)):
        compare(cache, kval, vval, table, q, cu, lens, 2 * G, 0.1, w, s)


def test_rows_between_sequences():
    """Offsets that leave gaps: rows of no sequence stay as they were; offsets out of range leave a sequence out."""
    page, d, kv, G = 16, 64, 2, 2
    cache, kval, vval, table, q, cu, lens = case(12, [(400, 400), (50, 500), (20, 20)], kv, G, d, page, "bf16")
    for c in ([10, 60, 60, 300], [0, 50, 471, 480], [0, 50, 40, 400], [-4, 50, 90, 100], [5, 2 ** 31 - 1, -2 ** 31, 7]):
        out = torch.full((q.shape[0], 4 * d), 3.0, dtype=torch.bfloat16, device="cuda")
        run(cache, table, q, c, lens, 4, 0.1, out=out)
        want, _, bound, covered = S.chunk_want(q, kval, vval, table, c, lens, page, 0.1, 4)
        assert (out[~covered] == 3).all(), c
        if c == [0, 50, 40, 400]:                          # rows 40 .. 49 are in two sequences: not defined
            covered[40:50] = False
        R.check(out.view(want.shape)[covered], want[covered], bound[covered], c)


def test_lengths_past_the_table_are_clamped():
    """A length that passes the block table's reach counts as that reach, as in lora_attn_decode."""
    page, d, G = 16, 128, 4
    cache, kval, vval, table, q, cu, lens = case(30, [(20, 160), (7, 96)], 1, G, d, page, "int8")
    got = run(cache, table, q, cu, [1 << 30, 96], G, 0.1)
    want = run(cache, table, q, cu, [160, 96], G, 0.1)
    assert torch.equal(got, want)
    assert (run(cache, table, q, cu, [-5, 0], G, 0.1) == 0).all()


def test_stream_graph_and_same_bits():
    """A captured call replays with new offsets and lengths on another stream; the workspace serves call after call."""
    page, d, kv, G = 16, 128, 2, 4
    cache, kval, vval, table, q, cu, lens = case(14, [(300, 1200), (90, 800), (5, 3000)], kv, G, d, page, "bf16")
    ct, lt, ws = A.int32(cu), A.int32(lens), workspace()
    first = run(cache, table, q, ct, lt, 8, 0.1, ws=ws)
    for _ in range(10):
        assert torch.equal(run(cache, table, q, ct, lt, 8, 0.1, ws=ws), first)
    out = torch.zeros_like(first)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        run(cache, table, q, ct, lt, 8, 0.1, ws=ws, out=out, stream=s)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first)
    for c, ls in (([0, 1, 2, 395], [1200, 1, 2999]), ([0, 395, 395, 395], [1000, 5, 5]), ([0, 0, 0, 395], [0, 0, 395])):
        ct.copy_(A.int32(c))
        lt.copy_(A.int32(ls))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        want, _, bound, _ = S.chunk_want(q, kval, vval, table, c, ls, page, 0.1, 8)
        R.check(out.view(want.shape), want, bound, c)


def test_one_row_is_the_decode_call():
    """Chunks of one row over the same cache as lora_attn_decode: within the bound of each other's."""
    page, d, kv, G = 16, 128, 2, 4
    nl = [(1, m) for m in (1, 100, 5000, 64)]
    cache, kval, vval, table, q, cu, lens = case(40, nl, kv, G, d, page, "e4m3")
    want, _, bound, _ = S.chunk_want(q, kval, vval, table, cu, lens, page, 0.1, 8, rounded=ROUNDED)
    q = q.contiguous()
    for got in (run(cache, table, q, cu, lens, 8, 0.1), A.run_decode(q, cache, table, A.int32(lens), 8, 0.1)):
        R.check(got.view(want.shape), want, bound)


@pytest.mark.parametrize("fmt", FMTS)
def test_as_many_sequences_as_a_call_takes(fmt):
    """8192 sequences, many threads' worth of the plan's: every one as its like among seven."""
    nl = [(1, 1), (2, 40), (0, 130), (1, 0), (3, 77), (1, 260), (2, 1)]
    cache, kval, vval, table, q, cu, lens = case(50, nl, 1, 2, 64, 16, fmt)
    out, _, bound, _ = S.chunk_want(q, kval, vval, table, cu, lens, 16, 0.1, 2, rounded=ROUNDED if fmt != "bf16" else 0.0)
    if fmt != "bf16":
        bound = bound + f16_floor(vval, lens)
    like = [b * 5 % 7 for b in range(8192)]
    rows = torch.tensor([r for b in like for r in range(cu[b], cu[b + 1])], device="cuda")
    got = run(cache, table[torch.tensor(like, device="cuda")].contiguous(), q[rows], starts([nl[b][0] for b in like]), [lens[b] for b in like], 2, 0.1)
    R.check(got.view(len(rows), 2, 64), out[rows], bound[rows], "8192")


def test_two_calls_at_once():
    """On two streams, each with a workspace of its own: the bits that they give one after another."""
    data = [case(60 + i, [(300 + i, 3000), (5, 700)], 2, 4, 128, 16, "bf16") for i in range(2)]
    apart = [run(c, t, q, cu, lens, 8, 0.1) for c, _, _, t, q, cu, lens in data]
    streams, spaces, outs = [torch.cuda.Stream() for _ in range(2)], [workspace() for _ in range(2)], [torch.full_like(a, float("nan")) for a in apart]
    ints = [(A.int32(d[5]), A.int32(d[6])) for d in data]
    torch.cuda.synchronize()
    for _ in range(5):
        for (c, _, _, t, q, _, _), (cu, lens), s, ws, o in zip(data, ints, streams, spaces, outs):
            run(c, t, q, cu, lens, 8, 0.1, ws=ws, out=o, stream=s)
    torch.cuda.synchronize()
    for a, o in zip(apart, outs):
        assert torch.equal(a, o)
