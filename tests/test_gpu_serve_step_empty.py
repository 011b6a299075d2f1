"""Calls of the example layer in which a sequence has no rows (-m gpu)."""
from __future__ import annotations

import torch
import pytest

from gather_lora_gb300 import serve_step
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu


def test_a_sequence_without_rows():
    """A prompt of no rows among others, new or after a first chunk: the others' results are the same bits."""
    require_gpu()
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(30, 256, generator=g, device="cuda").bfloat16()
    slot = torch.tensor([0] * 20 + [1] * 10, dtype=torch.int32, device="cuda")
    a, b = (serve_step.AttentionLayer(hidden=256, q_heads=4, kv_heads=2, head_dim=64, cache="int8", pages=20, seed=5) for _ in range(2))
    assert torch.equal(a.prefill(x, [0, 9, 1], [20, 0, 10], slot), b.prefill(x, [0, 1], [20, 10], slot))
    assert torch.equal(a.prefill(x[:5], [9, 0, 1], [0, 5, 0], slot[:5]), b.prefill(x[:5], [0], [5], slot[:5]))
    assert a.lengths == {0: 25, 9: 0, 1: 10}
    assert a.prefill(x[:0], [0, 9], [0, 0], slot[:0]).shape == (0, 256)
