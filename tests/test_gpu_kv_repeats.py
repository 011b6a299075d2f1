"""lora_kv_write with a slot named more than once (-m gpu): what that slot holds is not defined, all others are."""
from __future__ import annotations

import pytest
import torch

import attn_util as A
from gather_lora_gb300 import lib as L
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "int8"])
@pytest.mark.parametrize("n", [40, 9000])
def test_repeated_slots_touch_no_other(fmt, n):
    require_gpu()
    kv, d, page, pages = 2, 64, 16, 700
    g = A.gen(n)
    x = A.randn(g, n, 2 * kv * d)
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:n].clone()
    twice = slots[7].item()
    slots[11:n:3] = twice
    once = torch.ones(n, dtype=torch.bool, device="cuda")
    once[7], once[11:n:3] = False, False

    def write(rows):
        p = A.pool(pages, kv, page, d, fmt, fill=0x5A)
        s = [None, None] if fmt == "bf16" else [torch.full((pages, kv, page), 7.0, device="cuda") for _ in range(2)]
        k, v = x[rows, :kv * d].contiguous(), x[rows, kv * d:].contiguous()
        L.lora_kv_write(k, kv * d, v, kv * d, slots[rows].contiguous(), k.shape[0], L.KvCache(*p, *s))
        keep = torch.ones(pages * page, dtype=torch.bool, device="cuda")
        keep[twice] = False
        held = [t.view(torch.uint8).transpose(1, 2).reshape(pages * page, -1)[keep] for t in p]
        return held + [t.transpose(1, 2).reshape(pages * page, -1)[keep] for t in s if t is not None]
    every = write(torch.arange(n, device="cuda"))
    for a, b in zip(every, write(once.nonzero().flatten())):
        assert torch.equal(a, b)
