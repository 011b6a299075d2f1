"""The example layer's bookkeeping on the CPU: slots, pages, refusals. No kernel is launched here."""
from __future__ import annotations

import pytest
import torch

from gather_lora_gb300 import serve_step


def layer(**kw):
    return serve_step.AttentionLayer(hidden=64, q_heads=2, kv_heads=1, head_dim=64, device="cpu", **dict(dict(pages=6, page_size=4), **kw))


def test_slots_are_int64_whatever_the_count():
    """A sequence without rows adds no slots and leaves the others' type alone (the cache kernels read int64)."""
    lay = layer()
    none, some = lay._slots(0, 0, 0), lay._slots(1, 0, 5)
    assert none.dtype == some.dtype == torch.int64 and none.numel() == 0
    slots = torch.cat([none, some])
    assert slots.dtype == torch.int64
    pages = lay.tables[1]
    assert slots.tolist() == [pages[t // 4] * 4 + t % 4 for t in range(5)]
