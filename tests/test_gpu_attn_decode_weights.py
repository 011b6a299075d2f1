"""Decode over 8-bit caches against the bound for weights of 11 significant bits (-m gpu)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import attn_refs as R
import attn_util as A
import weight_refs as W
from gather_lora_gb300 import lib as L
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kv,G", [(2, 1), (2, 4), (1, 8), (2, 16), (1, 40)])
def test_weights_over_8_bit_caches(fmt, d, kv, G):
    require_gpu()
    lens, page = [1, 2, 3, 5, 9, 40, 200], 16
    q, rows = W.case(kv * 100 + G + d, fmt, kv, G, d, lens)
    want, bound = W.want(q, rows, 0.1)
    g = A.gen(1)
    num = sum(-(-n // page) for n in lens) + 1
    table = A.block_table(g, lens, page, num)
    pages = A.pool(num, kv, page, d, fmt)
    scales = [torch.zeros(num, kv, page, device="cuda") for _ in range(2)]
    for b, n in enumerate(lens):
        t = torch.arange(n, device="cuda")
        pg, sl = table[b].long()[t // page], t % page
        for i in range(2):
            pages[i][pg, :, sl] = torch.from_numpy(rows[b][2 * i]).cuda().float().to(R.DTYPE[fmt])
            scales[i][pg, :, sl] = torch.from_numpy(np.ascontiguousarray(rows[b][2 * i + 1])).cuda()
    x = torch.from_numpy(q).cuda().bfloat16().view(len(lens), -1)
    out = A.run_decode(x, L.KvCache(*pages, *scales), table, A.int32(lens), kv * G, 0.1)
    R.check(out.view(want.shape), torch.from_numpy(want).cuda(), torch.from_numpy(bound).cuda())
