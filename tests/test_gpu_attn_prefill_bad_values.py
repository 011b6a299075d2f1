"""Prefill attention over data that is not finite (-m gpu): the rows that see it get what the formula gives, all
others keep their results to the bit, at about the price of clean data and with the device status at zero."""
from __future__ import annotations

import itertools

import pytest
import torch

import attn_refs as R
import attn_util as A
from gather_lora_gb300 import lib as L
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    require_gpu()
    L.lora_read_device_status(clear=True)
    yield
    assert L.lora_read_device_status(clear=True) == 0


def case(seed, qk, kv, G, d, spread=1.0):
    g = A.gen(seed)
    cu_q, cu_k = ([0] + list(itertools.accumulate(x)) for x in zip(*qk))
    q = A.randn(g, cu_q[-1], kv * G * d, spread=spread)
    k, v = (A.randn(g, cu_k[-1], kv * d, spread=s) for s in (spread, 1.0))
    return q, k, v, cu_q, cu_k


def compare(q, k, v, cu_q, cu_k, kv, G, d, scale):
    """Finite results within the bound, infinities and NaN where the formula has them."""
    H = kv * G
    lse = torch.full((q.shape[0], H), 5.0, device="cuda")
    out = A.run_prefill(q, k, v, A.int32(cu_q), A.int32(cu_k), H, kv, scale, lse=lse)
    want, wl, bound, covered = A.prefill_want(q, k, v, cu_q, cu_k, H, kv, scale)
    got, want, bound = out.view(want.shape)[covered].double(), want[covered], bound[covered]
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got[torch.isinf(want)], want[torch.isinf(want)])
    off = ((got - want).abs() - bound)[fine]
    assert torch.isfinite(got[fine]).all() and (off.numel() == 0 or off.max().item() <= 0), off.max().item()
    mag = scale * d * q.double().abs().amax() * k.double().abs().nan_to_num(0, 0, 0).amax()
    R.check_lse(lse[covered], wl[covered], mag, "lse")
    return out


SHAPES = [(1, 1, [(300, 300), (70, 90), (129, 500)]), (2, 4, [(200, 200), (100, 333), (40, 40)]), (1, 8, [(257, 257), (17, 640)]),
          (1, 130, [(5, 260), (3, 3)]), (2, 1, [(130, 70), (60, 60)]),                    # rows without keys among them
          (1, 4, [(6, 3000), (4, 2500)]), (2, 8, [(33, 4000)])]                            # keys split over a cluster


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kv,G,qk", SHAPES)
def test_single_values_of_v(kv, G, qk, d):
    """One element of a V row, at places along each sequence's end (the key tiles that rows see in part) and
    elsewhere: infinite results in that dimension alone, for the rows that see the key, of that key-value head.
    Scores are small, so that no weight underflows."""
    q, k, v, cu_q, cu_k = case(kv * 7 + G + d, qk, kv, G, d, spread=0.3)
    r = torch.Generator().manual_seed(G)
    for b, (lq, lk) in enumerate(qk):
        for value in (INF, -INF, INF):
            at = cu_k[b] + max(0, lk - 1 - int(torch.randint(0, max(1, min(lk, lq + 20)), (1,), generator=r)))
            v[at, int(torch.randint(0, kv * d, (1,), generator=r))] = value
    compare(q, k, v, cu_q, cu_k, kv, G, d, 0.1)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kv,G,qk", SHAPES)
def test_a_sequence_that_is_not_finite_keeps_to_itself(kv, G, qk, d):
    """All of one sequence's K and V is NaN: its rows that see a key are NaN; the sequences behind it keep their bits, and
    those before it, whose last key tile may hold some of its rows, their values (one BF16 step, as sums in fp32
    may run in another order)."""
    q, k, v, cu_q, cu_k = case(kv * 11 + G + d, qk, kv, G, d)
    run = lambda: A.run_prefill(q, k, v, A.int32(cu_q), A.int32(cu_k), kv * G, kv, 0.1)
    clean = run()
    for b, (lq, lk) in enumerate(qk):
        keys = slice(cu_k[b], cu_k[b + 1])
        old = k[keys].clone(), v[keys].clone()
        k[keys], v[keys] = NAN, NAN
        got = run()
        for x in range(len(qk)):
            rows = slice(cu_q[x], cu_q[x + 1])
            if x > b:
                assert torch.equal(got[rows], clean[rows])
            elif x < b:
                assert torch.isfinite(got[rows]).all()
                assert ((got[rows].double() - clean[rows].double()).abs() <= clean[rows].double().abs() * 2 ** -7 + 1e-5).all()
            else:
                some = cu_q[x] + max(0, lq - lk)
                assert torch.isnan(got[some:cu_q[x + 1]]).all() and (got[cu_q[x]:some] == 0).all()
        k[keys], v[keys] = old


def test_values_near_the_largest():
    """V near 2^119 and maxima that rise by less than 2^8 from tile to tile: weights never pass 1, so sums that fit
    fp32 by the formula stay finite."""
    for d, G in ((64, 2), (128, 4)):
        q, k, v, cu_q, cu_k = case(3, [(600, 600), (9, 2500)], 1, G, d)
        q = torch.ones_like(q)
        k = (k.float() * 0.01 + torch.arange(k.shape[0], device="cuda")[:, None] // 128 * (3.0 / d)).bfloat16()
        v = ((v.float().abs() + 1) * 2.0 ** 118).bfloat16()
        compare(q, k, v, cu_q, cu_k, 1, G, d, 1.0)


def clock(f, n=5):
    f()
    at = [torch.cuda.Event(enable_timing=True) for _ in range(2 * n)]
    for i in range(n):
        at[2 * i].record()
        f()
        at[2 * i + 1].record()
    torch.cuda.synchronize()
    return min(at[2 * i].elapsed_time(at[2 * i + 1]) for i in range(n))


@pytest.mark.parametrize("where", ["first key", "last keys", "everywhere"])
def test_the_price_of_bad_values(where):
    """A prompt of 8192: NaN at its first key is a part of every result and costs next to nothing. NaN in key tiles
    that rows see in part costs those tiles a scalar pass: never more than a few times the call."""
    kv, G, d, n = 4, 8, 128, 8192
    q, k, v, cu_q, cu_k = case(1, [(n, n)], kv, G, d)
    cq, ck, out = A.int32(cu_q), A.int32(cu_k), torch.empty_like(q)
    run = lambda: A.run_prefill(q, k, v, cq, ck, kv * G, kv, d ** -0.5, out=out)
    clean = clock(run)
    rows = {"first key": slice(0, 1), "last keys": slice(n - 100, n), "everywhere": slice(0, n)}[where]
    k[rows], v[rows] = NAN, NAN
    t = clock(run)
    assert torch.isnan(out[rows.start:]).all() and torch.isfinite(out[:rows.start]).all()
    print(f"{where}: {t:.3f} ms against {clean:.3f}")
    assert t < (10 if where == "everywhere" else 2) * clean, (t, clean)


@pytest.mark.parametrize("others", [2, 120])
@pytest.mark.parametrize("bad", ["early", "next"])
def test_a_long_context_does_not_hold_up_the_rest(others, bad):
    """64 rows after a million keys, not finite from an early key on, or with a sequence that is not finite behind it (which
    shares the last key tile): the other sequences of the call get their results. With few sequences
    the keys are split over a cluster, with many they are not."""
    kv, G, d, long = 1, 4, 64, (1 << 20) + 37
    qk = [(64, long), (64, 200)] + [(50, 50 + i) for i in range(others - 1)]
    q, k, v, cu_q, cu_k = case(2, qk, kv, G, d, spread=0.5)
    run = lambda: A.run_prefill(q, k, v, A.int32(cu_q), A.int32(cu_k), G, kv, 0.1)
    clean = run()
    assert torch.isfinite(clean).all()
    rows, hurt = (slice(5, long), slice(0, 64)) if bad == "early" else (slice(cu_k[1], cu_k[2]), slice(64, 128))
    k[rows], v[rows] = NAN, NAN
    got = run()
    assert L.lora_read_device_status(clear=True) == 0
    assert torch.isnan(got[hurt]).all()
    keep = torch.ones(q.shape[0], dtype=torch.bool, device="cuda")
    keep[hurt] = False
    assert torch.isfinite(got[keep]).all()
    assert (got[keep].double() - clean[keep].double()).abs().max() <= 2 ** -7 * clean[keep].abs().max()
    assert torch.equal(got[128:], clean[128:])
