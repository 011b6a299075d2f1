"""lora_attn_chunk over 8-bit caches where one token has nearly all of a row's weight and V is 0 there in most elements: what the
others with weights of 2^-14 .. 2^-26 add is as exact whichever way the one's tile is taken (-m gpu)."""
from __future__ import annotations

import math

import pytest
import torch

import attn_refs as R
import attn_util as A
import step_refs as S
import test_gpu_attn_chunk as C
from gather_lora_gb300 import lib as L
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    require_gpu()
    L.lora_read_device_status(clear=True)
    yield
    assert L.lora_read_device_status(clear=True) == 0


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("d,page", [(64, 16), (128, 16), (128, 20), (64, 1)])
@pytest.mark.parametrize("n,m,at", [(1, 1500, 1499), (1, 1500, 3), (3, 1500, 1490), (200, 1500, 1200), (1, 300, 298)])
def test_beside_one_large_weight(fmt, d, page, n, m, at):
    """Token `at` has a score `gap` above all others'; its V is 1 in the first element and 0 elsewhere, the others' V is 1 and -1 by
    elements, of magnitudes by tokens."""
    kv, num, scale = 1, -(-m // page) + 1, 0.1
    g = A.gen(m + at)
    table = A.block_table(g, [m], page, num)
    q = torch.ones(n, d, dtype=torch.bfloat16, device="cuda")
    for gap in (9.7, 13.0, 15.25, 16.6, 18.0):
        k = torch.zeros(num, kv, page, d, device="cuda")
        v = torch.where(torch.arange(d, device="cuda") % 2 == 0, 1.0, -1.0) * 2.0 ** -torch.randint(0, 3, (num, kv, page, 1), generator=g, device="cuda")
        pg, sl = C.place(table, page, 0, at)
        k[pg, 0, sl] = gap / (scale * d)
        v[pg, 0, sl] = 0
        v[pg, 0, sl, 0] = 1
        cache, kval, vval = A.cache_from_values(k.bfloat16(), v.bfloat16(), fmt)
        assert math.isclose(scale * kval[pg, 0, sl].sum().item(), gap, rel_tol=0.01)
        C.compare(cache, kval, vval, table, q, [0, n], [m], 1, scale)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("page", [16, 20])
def test_in_whole_contexts(fmt, page):
    """The same in as many sequences as give a CTA whole ones. The token is in the first tile, which is taken token by token, as the
    scales in it are far apart; the tiles behind it are not."""
    d, num, scale, batch, m = 64, -(-1500 // page) + 1, 0.1, 400, 1500
    g = A.gen(page)
    table = A.block_table(g, [m], page, num)
    q = torch.ones(batch, d, dtype=torch.bfloat16, device="cuda")
    for gap in (13.0, 14.9, 15.6, 16.6):
        k, v = torch.zeros(num, 1, page, d, device="cuda"), torch.ones(num, 1, page, d, device="cuda")
        pg, sl = C.place(table, page, 0, [3, 5])
        k[pg[:1], 0, sl[:1]], v[pg[:1], 0, sl[:1]], v[pg[1:], 0, sl[1:]] = gap / (scale * d), 0, 2.0 ** -14
        v[pg[:1], 0, sl[:1], 0] = 1
        cache, kval, vval = A.cache_from_values(k.bfloat16(), v.bfloat16(), fmt)
        out = C.run(cache, table.repeat(batch, 1), q, list(range(batch + 1)), [m] * batch, 1, scale)
        want, _, bound, _ = S.chunk_want(q[:1], kval, vval, table, [0, 1], [m], page, scale, 1, rounded=C.ROUNDED)
        R.check(out.view(batch, 1, d), want.expand(batch, 1, d), (bound + C.f16_floor(vval, [m])).expand(batch, 1, d), gap)
