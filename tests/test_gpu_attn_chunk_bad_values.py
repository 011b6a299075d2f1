"""Elements of V that are not finite, in tiles that only the later rows of an item see, where the item is shared out over
several CTAs: the rows that see them get them, the others do not, and every call gives the same bits (-m gpu)."""
from __future__ import annotations

import pytest
import torch

import attn_util as A
import step_refs as S
import test_gpu_attn_chunk as C
from gather_lora_gb300 import lib as L
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    require_gpu()
    L.lora_read_device_status(clear=True)
    yield
    assert L.lora_read_device_status(clear=True) == 0


def put(cache, vval, page, table, b, head, t, e, bad):
    """V's element e of token t and head `head` becomes `bad` (E4M3: its NaN; INT8: the token's scale becomes NaN, all of it)."""
    pg, sl = (x.item() for x in C.place(table, page, b, t))
    _, v, _, vs = cache.tensors
    if v.dtype == torch.bfloat16:
        v[pg, head, sl, e] = vval[pg, head, sl, e] = bad
    elif v.dtype == torch.int8:
        vs[pg, head, sl] = NAN
        vval[pg, head, sl] = NAN
    else:
        v.view(torch.uint8)[pg, head, sl, e] = 0x7F
        vval[pg, head, sl, e] = NAN


def same_everywhere(data, h, scale, window, sinks):
    cache, kval, vval, table, q, cu, lens = data
    page, coded = cache.struct.page_size, cache.struct.format != L.KV_BF16
    ws = C.workspace()
    out = C.run(cache, table, q, cu, lens, h, scale, window, sinks, ws=ws)
    want, _, bound, _ = S.chunk_want(q, kval, vval, table, cu, lens, page, scale, h, window, sinks, rounded=C.ROUNDED if coded else 0.0)
    got = out.view(want.shape).double()
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"NaN lost or made: {(torch.isnan(got) != torch.isnan(want)).sum().item()}"
    assert torch.equal(got[torch.isinf(want)], want[torch.isinf(want)]) and torch.equal(torch.isinf(got), torch.isinf(want))
    fine = torch.isfinite(want)
    # (where V is not finite among a row's tokens its bound is not either)
    held = fine & torch.isfinite(bound)
    floor = C.f16_floor(vval, lens) if coded else 0.0
    assert ((got - want).abs()[held] <= (bound + floor)[held]).all()
    for _ in range(5):
        assert torch.equal(C.run(cache, table, q, cu, lens, h, scale, window, sinks, ws=ws).view(torch.int16), out.view(torch.int16))
    return got, fine


@pytest.mark.parametrize("fmt", C.FMTS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 20])                             # (20: no multiple of 8 slots, read token by token)
@pytest.mark.parametrize("kv", [5, 38])
def test_tiles_of_the_later_rows_alone(fmt, d, page, kv):
    """256 rows after 128 tokens, one head a group: two row tiles of 128 rows, of three key tiles the last is seen by the second
    row tile alone. 5 heads over 152 CTAs give parts that hold nothing but it."""
    n, m = 256, 384
    data = C.case(kv + d, [(n, m)], kv, 1, d, page, fmt)
    cache, kval, vval, table, q, cu, lens = data
    clean = C.run(cache, table, q, cu, lens, kv, 0.1).view(n, kv, d)
    bad = [INF, NAN, -INF]
    for head in range(kv):
        for x, t in enumerate((257 + head % 100, 383 - head % 20)):
            put(cache, vval, page, table, 0, head, t, (7 * head + 31 * x) % d, bad[(head + x) % 3])
    got, fine = same_everywhere(data, kv, 0.1, S.EVERY, 0)
    assert not fine.all()
    # rows before the tokens are as they were, to the bit
    before = torch.arange(n, device="cuda") + (m - n) < 257
    assert torch.equal(got[before], clean[before].double())


@pytest.mark.parametrize("fmt", C.FMTS)
@pytest.mark.parametrize("d,kv,G,page,window,sinks", [(64, 5, 1, 32, 600, 16), (128, 3, 2, 16, S.EVERY, 0), (64, 2, 5, 7, 300, 0)])
def test_last_tiles_of_windows_and_packed_chunks(fmt, d, kv, G, page, window, sinks):
    """Bad values among each chunk's last tokens and at its window's beginning, over item ends of every kind."""
    nl = [(300, 1500), (256, 384), (129, 1000), (40, 40), (257, 2049)]
    data = C.case(d + kv + G, nl, kv, G, d, page, fmt)
    cache, kval, vval, table, q, cu, lens = data
    for b, (n, m) in enumerate(nl):
        for head in range(kv):
            for x, t in enumerate((m - 1 - head % 5, m - n // 3, max(0, m - n - window + n // 2) if window < m else m - 3)):
                put(cache, vval, page, table, b, head, t, (5 * head + 17 * x + b) % d, (INF, -INF, NAN)[(b + x) % 3])
    same_everywhere(data, kv * G, 0.1, window, sinks)


def spoil_scales(cache, page, table, b, t, head, bad):
    pg, sl = C.place(table, page, b, t)
    cache.tensors[3][pg, head, sl] = bad


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("d,G,page", [(64, 1, 16), (128, 4, 16), (128, 2, 20)])
@pytest.mark.parametrize("bad", [NAN, INF, -INF])
@pytest.mark.parametrize("spread", [1.0, 1e4])                         # (1e4: scales of a tile too far apart for one factor)
def test_the_sum_of_the_weights_does_not_go_by_v(fmt, d, G, page, bad, spread):
    """A V scale that is not finite, in tokens that all rows see and in tokens that some see: lse is what it is without V,
    the rows that see the token are NaN in that head and the others are as they were."""
    kv, nl = 2, [(200, 500), (3, 130), (300, 3000)]
    cache, kval, vval, table, q, cu, lens = C.case(d + G, nl, kv, G, d, page, fmt)
    cache.tensors[3][:, :, ::3] *= spread
    vval[:, :, ::3] *= spread
    h, clean = kv * G, C.run(cache, table, q, cu, lens, kv * G, 0.1).view(-1, kv, G, d)
    _, wl, _, _ = S.chunk_want(q, kval, vval, table, cu, lens, page, 0.1, h, rounded=C.ROUNDED)
    hit = torch.zeros(q.shape[0], kv, dtype=torch.bool, device="cuda")
    for b, (n, m) in enumerate(nl):
        for head, at in ((0, [m - 1, m - n // 2 - 1]), (1, [10] if b else [m - 150])):
            spoil_scales(cache, page, table, b, at, head, bad)
            hit[cu[b]:cu[b + 1], head] = S.seen(n, m, S.EVERY, 0)[:, at].any(1)
    lse = torch.full((q.shape[0], h), 5.0, device="cuda")
    out = C.run(cache, table, q, cu, lens, h, 0.1, lse=lse).view(-1, kv, G, d)
    assert torch.isnan(out[hit]).all() and torch.equal(out[~hit], clean[~hit])
    mag = 0.1 * d * q.double().abs().amax() * kval.abs().amax()
    C.R.check_lse(lse, wl, mag * (1 + C.ROUNDED * 2 ** 24 / 140), "lse")


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("page", [16, 20])
def test_a_scale_that_is_not_finite_among_zeros(fmt, page):
    """All other scales of V are 0: the rows that see the one token are not finite, the others are 0."""
    n, m, d = 50, 400, 64
    cache, kval, vval, table, q, cu, lens = C.case(3, [(n, m)], 2, 2, d, page, fmt)
    cache.tensors[3][:] = 0
    for head, t in ((0, 60), (1, m - 20)):
        spoil_scales(cache, page, table, 0, [t], head, INF)
    out = C.run(cache, table, q, cu, lens, 4, 0.1).view(n, 2, 2, d)
    assert not torch.isfinite(out[:, 0]).any()
    assert not torch.isfinite(out[n - 20:, 1]).any() and (out[:n - 20, 1] == 0).all()
