"""Head norms without a rotation: positions and their stride are ignored (rotary_dim 0)."""
from __future__ import annotations

import ctypes
import os

import pytest
import torch

import attn_util as A
import step_refs as S
import test_gpu_rope as T
from gather_lora_gb300 import lib as L
from gpu_util import require_gpu
from test_attn_abi_cpu import _cache


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not os.path.exists(L.LIB_PATH):
        from gather_lora_gb300 import build
        build.build()
    L.load()


def test_the_stride_is_ignored():
    """On the host, in calls without rows: no stride is refused without a rotation, and a short one is with it."""
    for rotary, code in ((0, 0), (8, -3)):
        r, c = ctypes.byref(L.Rope(128, rotary_dim=rotary).struct), ctypes.byref(_cache())
        assert L.load().lora_qk_rope(None, 1024, None, 1024, None, 512, None, 512, 0, 8, 4, r, None, -1, None, None, 1e-6, None) == code
        assert L.load().lora_kv_append(None, 1024, None, 1024, 8, None, 512, None, 512, None, 0, c, r, None, -1, None, None, 1e-6, None) == code


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_norms_without_positions(d):
    require_gpu()
    g, n, hq, hkv = A.gen(d), 37, 6, 2
    rows = A.randn(g, n, (hq + 2 * hkv) * d, spread=2.0)
    norm, rope = (1 + 0.3 * torch.randn(d, generator=g, device="cuda")).bfloat16(), L.Rope(d, rotary_dim=0)
    q, k = (torch.empty(n, h * d, dtype=torch.bfloat16, device="cuda") for h in (hq, hkv))
    L.lora_qk_rope(rows, rows.stride(0), q, hq * d, rows[:, hq * d:], rows.stride(0), k, hkv * d, n, hq, hkv, rope, None, 0, q_norm=norm, k_norm=norm, eps=T.EPS)
    for got, first, heads in ((q, 0, hq), (k, hq, hkv)):
        y, mag = S.turned(rows[:, first * d:(first + heads) * d].double().reshape(n, heads, d), torch.zeros(1, n), [], [], 0, False, norm, T.EPS)
        T.within(got, y, mag, heads)
    pages, sc, cache = T.fresh(5, hkv, 8, d, "bf16", "hnd")
    q2, slots = torch.empty_like(q), torch.randperm(40, generator=g, device="cuda")[:n].clone()
    L.lora_kv_append(rows, rows.stride(0), q2, hq * d, hq, rows[:, hq * d:], rows.stride(0), rows[:, (hq + hkv) * d:], rows.stride(0), slots, n, cache,
                     rope, None, 0, q_norm=norm, k_norm=norm, eps=T.EPS)
    assert torch.equal(q2, q) and torch.equal(pages[0][slots // 8, :, slots % 8].reshape(n, hkv * d), k)
