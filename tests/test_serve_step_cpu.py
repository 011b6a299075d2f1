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


def state(lay):
    return list(lay.free), {s: list(p) for s, p in lay.tables.items()}, dict(lay.lengths)


def test_too_few_pages_change_nothing():
    """6 pages of 4: a call that needs more is refused before any page is taken, for prompts, chunks and decode steps."""
    lay = layer()
    lay._slots(0, 0, 15)
    lay.lengths[0] = 15
    for seqs, counts in (([1], [9]), ([1, 2], [4, 5]), ([0, 1], [2, 5]), ([1, 2, 3], [1, 1, 1])):
        before = state(lay)
        x, slot = torch.zeros(sum(counts), 64, dtype=torch.bfloat16), torch.zeros(sum(counts), dtype=torch.int32)
        with pytest.raises(RuntimeError, match="pages are needed"):
            lay.prefill(x, seqs, counts, slot)
        assert state(lay) == before
    lay._slots(1, 0, 8)
    lay.lengths[0], lay.lengths[1] = 16, 8
    before = state(lay)
    with pytest.raises(RuntimeError, match="pages are needed"):
        lay.decode(torch.zeros(2, 64, dtype=torch.bfloat16), [0, 1], torch.zeros(2, dtype=torch.int32))
    assert state(lay) == before


def test_rows_that_do_not_fit_are_refused():
    lay = layer()
    x, slot = torch.zeros(5, 64, dtype=torch.bfloat16), torch.zeros(5, dtype=torch.int32)
    wide = torch.zeros(64, 5, dtype=torch.bfloat16).T
    for args in ((wide, [0], [5], slot), (x, [0], [4], slot), (x, [0, 1], [5], slot), (x, [0, 0], [2, 3], slot), (x, [0, 1], [6, -1], slot),
                 (x[:, :32], [0], [5], slot), (x, [0], [5], slot[:4]), (x, [0], [5], slot.long())):
        with pytest.raises(ValueError):
            lay.prefill(*args)
    for args in ((x, [0], slot), (x[:2], [3, 3], slot[:2])):
        with pytest.raises(ValueError):
            lay.decode(*args)
    assert state(lay) == (list(range(6)), {}, {})
