"""Sequences as long as a call takes, 2^31 - 64 tokens over a few pages named again and again: what stands at their end
is computed in 32 bits right up to it (-m gpu)."""
from __future__ import annotations

import pytest
import torch

import attn_refs as R
import attn_util as A
import test_gpu_attn_chunk as C
from gather_lora_gb300 import lib as L
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu
MOST = 2 ** 31 - 64


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    require_gpu()
    L.lora_read_device_status(clear=True)
    yield
    assert L.lora_read_device_status(clear=True) == 0


@pytest.mark.parametrize("fmt", C.FMTS)
@pytest.mark.parametrize("page,d", [(64 * 31, 64), (31 * 601, 128)])   # (pages by TMA; token by token. Both divide 2^31 - 64)
def test_rows_at_the_last_positions(fmt, page, d):
    g, kv, scale = A.gen(page + d), 2, 0.1
    cache, kval, vval = A.cache_from_values(A.randn(g, 3, kv, page, d), A.randn(g, 3, kv, page, d), fmt)
    table = torch.randint(0, 3, (1, MOST // page), generator=g, device="cuda", dtype=torch.int32)
    coded = fmt != "bf16"
    for n, G, length, window, sinks in ((1, 1, MOST, 300, 4), (1, 8, MOST, 130, 0), (100, 1, MOST, 300, 4), (200, 1, MOST, 257, 0),
                                        (256, 1, MOST, 90, 130), (33, 4, MOST - 1, 300, 4), (300, 2, MOST - 70, 500, 1)):
        h = kv * G
        guard = 300                                       # rows behind the sequence's, left as they are
        q = A.randn(g, n + guard, h * d)
        out = torch.full((n + guard, h * d), 3.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((n + guard, h), 5.0, device="cuda")
        C.run(cache, table, q, [0, n], [length], h, scale, window, sinks, out=out, lse=lse)
        assert (out[n:] == 3).all() and (lse[n:] == 5).all()
        t = torch.cat((torch.arange(sinks, device="cuda"), torch.arange(length - n - window, length, device="cuda")))
        p = torch.arange(length - n, length, device="cuda")[:, None]
        see = (t <= p) & ((t > p - window) | (t < sinks))
        pg, sl = table[0].long()[t // page], t % page
        both = [out[:n].view(n, h, d)]
        if n == 1:
            alone, ws = torch.empty(1, h * d, dtype=torch.bfloat16, device="cuda"), A.workspace()
            L.lora_attn_decode_window(q, h * d, alone, h * d, 1, h, scale, cache, table, table.stride(0), table.shape[1], A.int32([length]),
                                      window, sinks, ws, ws.numel())
            both.append(alone.view(1, h, d))
        for a in range(h):
            x, k, v = q[:n].double().view(n, h, d)[:, a], kval[pg, a // G, sl], vval[pg, a // G, sl]
            want, _, bound = R.attend(x, k, v, scale, see)
            if coded:                                     # (as tests/step_refs.py and tests/test_gpu_attn_chunk.py derive it)
                dz = C.ROUNDED * torch.where(see, scale * (x.abs() @ k.abs().T), 0.0).amax(1, keepdim=True)
                w = torch.softmax(torch.where(see, scale * (x @ k.T), -torch.inf), 1)
                bound = bound + (torch.expm1(2 * dz) + C.ROUNDED) * (w @ v.abs()) + 2.0 ** -32 * t.numel() * v.abs().amax()
            for got in both:
                R.check(got[:, a], want, bound, (n, G, length))
