"""The example layer (folds, cache, attention, output fold) against a plain 64-bit form of it (-m gpu)."""
from __future__ import annotations

import pytest
import torch

from gather_lora_gb300 import serve_step
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    require_gpu()


def test_the_example_agrees_with_itself():
    serve_step.main()


@pytest.mark.parametrize("kv,d", [(2, 64), (1, 128)])
def test_layer_against_64_bits(kv, d):
    """Prompts and decode steps with a BF16 cache. Every stage rounds to BF16 once or twice, each at most
    2^-8 of the value: projection, fold (two roundings inside), weights and result of the attention, output
    projection and fold; the whole differs by well under 8 * 2^-8 in the 2-norm."""
    lay = serve_step.AttentionLayer(hidden=256, q_heads=4, kv_heads=kv, head_dim=d, cache="bf16", pages=40, seed=3)
    g = torch.Generator(device="cuda").manual_seed(4)
    counts, steps, adapters = [1, 33, 50], 2, [1, -1, 3]
    rows = [torch.randn(n + steps, 256, generator=g, device="cuda").bfloat16() for n in counts]
    slot = [torch.full((r.shape[0],), a, dtype=torch.int32, device="cuda") for r, a in zip(rows, adapters)]
    y = lay.prefill(torch.cat([r[:n] for r, n in zip(rows, counts)]), [0, 1, 2], counts, torch.cat([t[:n] for t, n in zip(slot, counts)]))
    got = [[p] for p in y.split(counts)]
    for k in range(steps):
        y = lay.decode(torch.stack([r[n + k] for r, n in zip(rows, counts)]), [0, 1, 2], torch.stack([t[0] for t in slot]))
        for s in range(3):
            got[s].append(y[s:s + 1])

    def project(x, w, names, s):
        out, col = x @ w.double().T, 0
        for name in names:
            a, b = (t.double() for t in lay.adapters[name][:2])
            if adapters[s] >= 0:
                out[:, col:col + b.shape[1]] += 2.0 * (x @ a[adapters[s]].T) @ b[adapters[s]].T
            col += b.shape[1]
        return out
    for s, r in enumerate(rows):
        x = r.double()
        q, k, v = project(x, lay.w_qkv, "qkv", s).split(lay.widths, 1)
        n, G = x.shape[0], 4 // kv
        q, k, v = q.view(n, 4, d), k.view(n, kv, d).repeat_interleave(G, 1), v.view(n, kv, d).repeat_interleave(G, 1)
        z = torch.einsum("ihd,jhd->hij", q, k) * d ** -0.5
        z = z.masked_fill(torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1), -torch.inf)
        a = torch.einsum("hij,jhd->ihd", torch.softmax(z, -1), v).reshape(n, 4 * d)
        want = project(a, lay.w_o, "o", s)
        have = torch.cat(got[s]).double()
        off = ((have - want).norm() / want.norm()).item()
        assert off < 8 * 2.0 ** -8, (s, off)
    lay.release(1)
    assert 1 not in lay.tables and len(lay.free) == 40 - sum(len(p) for p in lay.tables.values())
