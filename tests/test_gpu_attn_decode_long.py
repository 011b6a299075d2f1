"""Contexts whose segment (sequence, key-value head, block of query heads) lies on every CTA of the GPU, so that
its parts join in two levels with more groups than one round of loads (-m gpu). Values drift along the context:
a part that is left out moves the mean of the rest by far more than the bound."""
from __future__ import annotations

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


def case(seed, lens, kv, G, d, page, fmt):
    g = A.gen(seed)
    need = [-(-n // page) for n in lens]
    num = sum(need) + 2
    table = A.block_table(g, lens, page, num)
    k, v = A.randn(g, num, kv, page, d, spread=0.3), A.randn(g, num, kv, page, d, spread=0.1)
    drift = torch.zeros(num, device="cuda")
    for b, m in enumerate(need):
        drift[table[b, :m].long()] = torch.linspace(-1, 1, m, device="cuda")
    v = (v.float() + drift[:, None, None, None]).bfloat16()
    cache, kval, vval = A.cache_from_values(k, v, fmt)
    return cache, kval, vval, table, A.randn(g, len(lens), kv * G * d)


def compare(lens, kv, G, d, page, fmt):
    cache, kval, vval, table, q = case(sum(lens), lens, kv, G, d, page, fmt)
    lse = torch.full((len(lens), kv * G), 5.0, device="cuda")
    ws, lt, scale = A.workspace(), A.int32(lens), d ** -0.5
    out = A.run_decode(q, cache, table, lt, kv * G, scale, ws=ws, lse=lse)
    want, wl, bound = A.decode_want(q, kval, vval, table, lens, page, scale, kv * G)
    R.check(out.view(want.shape), want, bound, "out")
    R.check_lse(lse, wl, scale * q.double().abs().amax() * kval.abs().amax() * d, "lse")
    for _ in range(20):                                      # the same bits, and the counters left at zero
        assert torch.equal(A.run_decode(q, cache, table, lt, kv * G, scale, ws=ws), out)
    assert int(ws[:3 * 512 * 4].count_nonzero()) == 0


@pytest.mark.parametrize("G", [1, 8, 16])
@pytest.mark.parametrize("fmt,d,n", [("bf16", 128, 17000), ("bf16", 128, 33000), ("bf16", 64, 70001), ("e4m3", 128, 40000),
                                     ("int8", 128, 40001), ("e4m3", 64, 70000), ("int8", 64, 70003)])
def test_one_sequence_on_every_cta(fmt, d, n, G):
    compare([n], 1, G, d, 64, fmt)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "int8"])
@pytest.mark.parametrize("lens", [[100000, 2000, 3000], [1, 100000, 0, 7], [40, 65000]])
def test_one_sequence_with_most_of_the_batch(fmt, lens):
    compare(lens, 1, 4, 128, 32, fmt)


def test_two_blocks_of_heads_share_the_grid():
    """17 query heads a group: two segments of one sequence, each on half of the CTAs."""
    compare([60000], 1, 17, 128, 64, "bf16")
