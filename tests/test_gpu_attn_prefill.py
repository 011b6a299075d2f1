"""Causal attention over packed sequences, against the 64-bit form within the bound derived in
tests/attn_refs.py (-m gpu)."""
from __future__ import annotations

import itertools

import pytest
import torch

import attn_refs as R
import attn_util as A
from gather_lora_gb300 import lib as L
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    require_gpu()
    L.lora_read_device_status(clear=True)
    yield
    assert L.lora_read_device_status(clear=True) == 0


def starts(ns):
    return [0] + list(itertools.accumulate(ns))


def case(seed, qk, kv, G, d, spread=1.0):
    """Packed q, k, v as parts of wider rows, and their offsets."""
    g = A.gen(seed)
    cu_q, cu_k = starts([a for a, _ in qk]), starts([b for _, b in qk])
    H = kv * G
    q = A.randn(g, cu_q[-1], (H + 2 * kv) * d + 16, spread=spread)[:, 8:8 + H * d]
    kvr = A.randn(g, cu_k[-1], 2 * kv * d + 8, spread=spread)
    return q, kvr[:, :kv * d], kvr[:, kv * d:2 * kv * d], cu_q, cu_k


def compare(q, k, v, cu_q, cu_k, kv, G, d, scale):
    H = kv * G
    lse = torch.full((q.shape[0], H), 5.0, device="cuda")
    out = A.run_prefill(q, k, v, A.int32(cu_q), A.int32(cu_k), H, kv, scale, lse=lse)
    want, wl, bound, covered = A.prefill_want(q, k, v, cu_q, cu_k, H, kv, scale)
    R.check(out.view(want.shape)[covered], want[covered], bound[covered], "out")
    if k.shape[0]:
        mag = scale * d * q.double().abs().nan_to_num(0, 0, 0).amax() * k.double().abs().nan_to_num(0, 0, 0).amax()
        R.check_lse(lse[covered], wl[covered], mag, "lse")
    return out


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kv,G", [(1, 1), (2, 2), (1, 3), (2, 5), (1, 7), (2, 8), (1, 16), (1, 48), (1, 130)])
def test_heads(d, kv, G):
    qk = [(1, 1), (33, 33), (150, 150), (0, 0), (7, 300)]
    compare(*case(kv * 1000 + G, qk, kv, G, d), kv, G, d, d ** -0.5)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300, 513])
def test_lengths(d, n):
    """One prompt of each length, alone, with a longer prefix, and with fewer keys than rows."""
    for qk in ([(n, n)], [(n, n + 1)], [(n, n + 130)], [(n, max(0, n - 1))], [(n, n // 2)], [(n, 1000)]):
        compare(*case(n, qk, 2, 4, d), 2, 4, d, 0.11)


@pytest.mark.parametrize("G", [1, 4, 8])
@pytest.mark.parametrize("d", [64, 128])
def test_packed(d, G):
    """Many sequences of different lengths in one call, empty ones and rows without keys among them."""
    r = torch.Generator().manual_seed(G)
    qk = [(int(a), int(a + max(0, b - 40))) for a, b in torch.randint(0, 200, (40, 2), generator=r).tolist()]
    qk[3], qk[10], qk[20], qk[39] = (0, 50), (64, 0), (100, 30), (0, 0)
    compare(*case(99 + d, qk, 2, G, d), 2, G, d, d ** -0.5)


@pytest.mark.parametrize("d,kv,G,qk", [(128, 1, 8, [(2100, 2100)]), (64, 4, 1, [(1030, 5000)]), (128, 2, 4, [(700, 700), (2048, 2048)])])
def test_long(d, kv, G, qk):
    compare(*case(5, qk, kv, G, d), kv, G, d, d ** -0.5)


@pytest.mark.parametrize("d", [64, 128])
def test_large_scores(d):
    """Scores that differ by thousands, maxima that rise along the keys."""
    q, k, v, cu_q, cu_k = case(6, [(300, 300), (100, 400)], 2, 4, d, spread=12.0)
    ramp = torch.linspace(0.1, 3.0, k.shape[0], device="cuda")[:, None]
    k = (k.float() * ramp).bfloat16()
    compare(q, k, v, cu_q, cu_k, 2, 4, d, 0.5)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf"), torch.finfo(torch.bfloat16).min])
@pytest.mark.parametrize("d", [64, 128])
def test_keys_that_are_not_seen_have_no_influence(d, bad):
    """Bad values in keys and values of later positions, of the next sequence and of rows between the
    sequences: rows that do not see them are as if they were not there."""
    kv, G = 1, 4
    q, k, v, cu_q, cu_k = case(8, [(200, 200), (70, 90), (40, 40)], kv, G, d)
    k, v = k.clone(), v.clone()
    for at in (137, 199, 200 + 60, 290 + 20):          # rows 137 and 199 of the first, ...
        k[at], v[at] = bad, bad
    H = kv * G
    out = A.run_prefill(q, k, v, A.int32(cu_q), A.int32(cu_k), H, kv, 0.1).view(-1, H, d)
    want, _, bound, _ = A.prefill_want(q, k, v, cu_q, cu_k, H, kv, 0.1)
    clean = torch.zeros(q.shape[0], dtype=torch.bool, device="cuda")
    clean[:137], clean[200:200 + 60 - 20], clean[270:290] = True, True, True
    R.check(out[clean], want[clean], bound[clean])
    assert torch.isfinite(out[clean]).all()
    if bad != bad:
        assert torch.isnan(out[137:200]).all() and torch.isnan(out[290:]).all()


@pytest.mark.parametrize("d", [64, 128])
def test_rows_between_sequences(d):
    """Offsets that leave gaps, in rows and keys; rows of no sequence stay as they were, and the gap
    keys (NaN) reach nobody. Offsets out of range leave a sequence out."""
    kv, G = 2, 2
    g = A.gen(12)
    q, k, v = A.randn(g, 400, 4 * d), A.randn(g, 500, 2 * d), A.randn(g, 500, 2 * d)
    cu_q, cu_k = [10, 60, 60, 300], [30, 95, 140, 420]
    k[:30], v[:30], k[420:], v[420:] = [float("nan")] * 4
    want, _, bound, covered = A.prefill_want(q, k, v, cu_q, cu_k, 4, kv, 0.1)
    out = torch.full((400, 4 * d), 3.0, dtype=torch.bfloat16, device="cuda")
    A.run_prefill(q, k, v, A.int32(cu_q), A.int32(cu_k), 4, kv, 0.1, out=out)
    assert (out[~covered] == 3).all()
    R.check(out.view(want.shape)[covered], want[covered], bound[covered])
    out.fill_(3.0)
    for bq, bk in (([0, 50, 401], [0, 50, 100]), ([0, 50, 100], [0, 50, 501]), ([0, 50, 100], [0, 50, 40]), ([0, 50, 100], [-4, 50, 90])):
        out.fill_(3.0)
        A.run_prefill(q, k, v, A.int32(bq), A.int32(bk), 4, kv, 0.1, out=out)
        bad_first = bk[0] < 0
        assert (out[50:] == 3).all() if not bad_first else (out[:50] == 3).all()


def test_same_bits_and_other_stream_and_graph():
    kv, G, d = 2, 4, 128
    q, k, v, cu_q, cu_k = case(14, [(300, 300), (90, 500)], kv, G, d)
    cq, ck = A.int32(cu_q), A.int32(cu_k)
    first = A.run_prefill(q, k, v, cq, ck, 8, kv, 0.1)
    for _ in range(10):
        assert torch.equal(A.run_prefill(q, k, v, cq, ck, 8, kv, 0.1), first)
    out = torch.zeros_like(first)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        A.run_prefill(q, k, v, cq, ck, 8, kv, 0.1, out=out, stream=s)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first)
    # the lengths are device data: other splits of the same rows
    cq.copy_(A.int32([0, 100, 390]))
    ck.copy_(A.int32([0, 100, 800]))
    graph.replay()
    torch.cuda.synchronize()
    want, _, bound, _ = A.prefill_want(q, k, v, [0, 100, 390], [0, 100, 800], 8, kv, 0.1)
    R.check(out.view(want.shape), want, bound)


def test_cached_prefix_end_to_end():
    """A prompt in two chunks through the cache equals the prompt in one call, within the bounds."""
    kv, G, d, page, n = 2, 4, 128, 16, 333
    g = A.gen(21)
    H = kv * G
    rows = A.randn(g, n, (H + 2 * kv) * d)
    q, k, v = rows[:, :H * d], rows[:, H * d:(H + kv) * d], rows[:, (H + kv) * d:]
    pages = A.pool(30, kv, page, d, "bf16")
    cache = L.KvCache(*pages)
    order = torch.randperm(30, generator=g, device="cuda")
    t = torch.arange(n, device="cuda")
    slots = order[t // page] * page + t % page
    L.lora_kv_write(k, k.stride(0), v, v.stride(0), slots, n, cache)
    kk, vv = (torch.empty(n, kv * d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    L.lora_kv_read(kk, kv * d, vv, kv * d, slots, n, cache)
    assert torch.equal(kk, k) and torch.equal(vv, v)
    part = A.run_prefill(q[200:], kk, vv, A.int32([0, n - 200]), A.int32([0, n]), H, kv, 0.1)
    want, _, bound, _ = A.prefill_want(q, k, v, [0, n], [0, n], H, kv, 0.1)
    R.check(part.view(-1, H, d), want[200:], bound[200:])
    # the last row as a decode step over the same cache
    table = order[None, :-(-n // page)].int().contiguous()
    last = A.run_decode(q[n - 1:], cache, table, A.int32([n]), H, 0.1)
    R.check(last.view(1, H, d), want[n - 1:], bound[n - 1:])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kv,G,qk", [
    (2, 4, [(5, 700)]), (1, 8, [(1, 2000)]), (2, 1, [(130, 1100)]), (1, 16, [(33, 9000)]), (3, 5, [(17, 4001)]),
    (1, 4, [(3, 5000), (40, 60), (2, 1), (70, 3000)]),        # parts without a key tile, a row without keys
    (2, 8, [(100, 1300), (0, 0), (9, 2600)]), (1, 130, [(2, 3000)]),
])
def test_few_rows_over_long_keys(d, kv, G, qk):
    """Shapes whose keys are split over the CTAs of a cluster and joined."""
    q, k, v, cu_q, cu_k = case(kv * 31 + G, qk, kv, G, d)
    out = compare(q, k, v, cu_q, cu_k, kv, G, d, d ** -0.5)
    again = A.run_prefill(q, k, v, A.int32(cu_q), A.int32(cu_k), kv * G, kv, d ** -0.5)
    assert torch.equal(out, again)


@pytest.mark.parametrize("d", [64, 128])
def test_few_rows_over_long_keys_bad_values(d):
    """Split keys: scores that differ by thousands between the parts; NaN in keys that rows do not see."""
    kv, G, qk = 1, 4, [(6, 3000), (4, 2500)]
    q, k, v, cu_q, cu_k = case(77, qk, kv, G, d, spread=8.0)
    ramp = torch.linspace(0.1, 2.0, k.shape[0], device="cuda")[:, None]
    k = (k.float() * ramp).bfloat16()
    compare(q, k, v, cu_q, cu_k, kv, G, d, 0.5)
    k, v = k.clone(), v.clone()
    k[2997:3000], v[2997:3000] = float("nan"), float("inf")     # rows 0 .. 2 of the first do not see them
    out = A.run_prefill(q, k, v, A.int32(cu_q), A.int32(cu_k), G, kv, 0.5).view(-1, G, d)
    want, _, bound, _ = A.prefill_want(q, k, v, cu_q, cu_k, G, kv, 0.5)
    keep = [0, 1, 2, 6, 7, 8, 9]
    R.check(out[keep], want[keep], bound[keep])
    assert torch.isnan(out[3:6]).all()
