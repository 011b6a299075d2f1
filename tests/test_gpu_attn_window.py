"""Attention of one new token per sequence that sees a sliding window and some first tokens, against the 64-bit form
within the bound derived in tests/attn_refs.py (-m gpu)."""
from __future__ import annotations

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


def case(seed, lens, kv, G, d, page, fmt, layout="hnd", extra=3):
    g = A.gen(seed)
    num = sum(-(-max(n, 0) // page) for n in lens) + extra
    cache, kval, vval = A.cache_from_values(A.randn(g, num, kv, page, d), A.randn(g, num, kv, page, d), fmt, layout)
    return cache, kval, vval, A.block_table(g, [max(n, 0) for n in lens], page, num), A.randn(g, len(lens), kv * G * d)


def run(q, cache, table, lens, h, scale, window, sinks, ws=None, out=None, lse=None, stream=None, max_pages=None):
    d = cache.struct.head_dim
    out = torch.full((q.shape[0], h * d), float("nan"), dtype=torch.bfloat16, device="cuda") if out is None else out
    ws = A.workspace() if ws is None else ws
    L.lora_attn_decode_window(q, q.stride(0), out, out.stride(0), q.shape[0], h, scale, cache, table, table.stride(0),
                              table.shape[1] if max_pages is None else max_pages, lens, window, sinks, ws, ws.numel(), lse=lse, stream=stream)
    return out


def compare(cache, kval, vval, table, q, lens, page, h, window, sinks, scale=0.1, ws=None):
    lse = torch.full((q.shape[0], h), 5.0, device="cuda")
    out = run(q, cache, table, A.int32(lens), h, scale, window, sinks, ws=ws, lse=lse)
    cu = list(range(len(lens) + 1))
    want, wl, bound, _ = S.chunk_want(q, kval, vval, table, cu, lens, page, scale, h, window, sinks)
    R.check(out.view(want.shape), want, bound, (window, sinks))
    R.check_lse(lse, wl, scale * q.shape[1] / h * q.double().abs().amax() * kval.abs().nan_to_num(0, 0, 0).amax(), "lse")
    return out


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d,kv,G,page", [(128, 2, 4, 16), (64, 3, 1, 20), (128, 1, 12, 64), (64, 2, 8, 1), (128, 1, 33, 8)])
def test_windows(fmt, d, kv, G, page):
    """Windows and first tokens of every kind against tiles of 16, 32 and 64 tokens: shorter and longer than the
    sequences, meeting, apart, inside one tile."""
    lens = [0, 1, 2, 15, 63, 64, 65, 129, 300, 777, -3]
    data = case(d + kv + G, lens, kv, G, d, page, fmt)
    for window, sinks in ((1, 0), (1, 1), (2, 3), (16, 0), (17, 15), (64, 64), (65, 1), (100, 200), (300, 4), (700, 0), (776, 1), (777, 0),
                          (5000, 3), (S.EVERY, 0), (3, 2 ** 31 - 1)):
        compare(*data[:5], lens, page, kv * G, window, sinks)


@pytest.mark.parametrize("fmt", FMTS)
def test_long_sequences_split_over_the_gpu(fmt):
    """Windows that many CTAs share, beside sequences that one takes."""
    lens = [40000, 33, 12000, 5]
    data = case(3, lens, 1, 4, 128, 64, fmt)
    ws = A.workspace()
    for window, sinks in ((9001, 4), (30000, 1000), (128, 0), (39000, 999)):
        a = compare(*data[:5], lens, 64, 4, window, sinks, ws=ws)
        assert torch.equal(a, run(data[4], data[0], data[3], A.int32(lens), 4, 0.1, window, sinks, ws=ws))


@pytest.mark.parametrize("fmt", FMTS)
def test_tokens_that_are_not_seen_have_no_influence(fmt):
    """Values between the first tokens and the window, and behind the sequence, that are NaN (and whose pages are not
    there): not read."""
    d, kv, G, page, n = 64, 2, 4, 16, 500
    cache, kval, vval, table, q = case(8, [n], kv, G, d, page, fmt)
    out = run(q, cache, table, A.int32([n]), kv * G, 0.1, 130, 21)
    want, _, bound, _ = S.chunk_want(q, kval, vval, table, [0, 1], [n], page, 0.1, kv * G, 130, 21)
    R.check(out.view(want.shape), want, bound)
    k_pages, v_pages, ks, vs = cache.tensors
    t = torch.arange(-(-n // page) * page, device="cuda")
    hide = ((t >= 21) & (t < n - 130)) | (t >= n)
    pg, sl = table[0].long()[t[hide] // page], t[hide] % page
    for x, s in ((k_pages, ks), (v_pages, vs)):
        if fmt == "bf16":
            x[pg, :, sl] = float("nan")
        else:
            x.view(torch.uint8)[pg, :, sl] = 0x7F
            s[pg, :, sl] = float("nan")
    assert torch.equal(run(q, cache, table, A.int32([n]), kv * G, 0.1, 130, 21), out)
    table = table.clone()
    table[0, 2:(n - 130) // page] = -1                     # pages that hold no visible token
    assert torch.equal(run(q, cache, table, A.int32([n]), kv * G, 0.1, 130, 21), out)
    table[0, (n - 130) // page + 2] = 10 ** 6              # a page inside the window that is not there: left out
    want, _, bound, _ = S.chunk_want(q, kval, vval, table, [0, 1], [n], page, 0.1, kv * G, 130, 21)
    R.check(run(q, cache, table, A.int32([n]), kv * G, 0.1, 130, 21).view(want.shape), want, bound)


def test_a_window_that_holds_everything_is_lora_attn_decode():
    lens = [900, 0, 33, 5000]
    cache, _, _, table, q = case(9, lens, 2, 4, 128, 16, "e4m3")
    for window in (5008, S.EVERY):
        assert torch.equal(run(q, cache, table, A.int32(lens), 8, 0.1, window, 0), A.run_decode(q, cache, table, A.int32(lens), 8, 0.1))


def test_graph_stream_and_shared_workspace():
    """A captured call replays over new lengths on another stream; calls of both kinds share a workspace in turn."""
    lens = [700, 64, 2000]
    cache, kval, vval, table, q = case(10, [2100] * 3, 2, 4, 128, 16, "bf16")
    lt, ws, out = A.int32(lens), A.workspace(), torch.zeros_like(q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        run(q, cache, table, lt, 8, 0.1, 300, 5, ws=ws, out=out, stream=s)
    for ls in (lens, [1, 2100, 0], [301, 305, 306]):
        lt.copy_(A.int32(ls))
        graph.replay()
        torch.cuda.synchronize()
        want, _, bound, _ = S.chunk_want(q, kval, vval, table, [0, 1, 2, 3], ls, 16, 0.1, 8, 300, 5)
        R.check(out.view(want.shape), want, bound, ls)
        full = A.run_decode(q, cache, table, lt, 8, 0.1, ws=ws)
        want, _, bound, _ = S.chunk_want(q, kval, vval, table, [0, 1, 2, 3], ls, 16, 0.1, 8)
        R.check(full.view(want.shape), want, bound, ls)
