"""Queries and keys normed and rotated, and appended to the paged cache, against the 64-bit form within the bounds
derived in tests/step_refs.py (-m gpu)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import attn_refs as R
import attn_util as A
import step_refs as S
from gather_lora_gb300 import lib as L
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu
EPS = 1e-5


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    require_gpu()


def rotation(d, rot, axes=1, inter=False, base=10000.0):
    freqs = [base ** (-2.0 * j / rot) for j in range(rot // 2)]
    axis = [(j * axes) // (rot // 2) for j in range(rot // 2)] if axes > 1 else [0] * (rot // 2)
    return freqs, axis, L.Rope(d, rotary_dim=rot, freqs=freqs, axis=axis if axes > 1 else None, interleaved=inter)


def positions(g, axes, n, far=100000):
    return torch.randint(0, far, (axes, n), generator=g, device="cuda", dtype=torch.int32)


def within(got, y, mag, what):
    """BF16 results within their bound (tests/step_refs.py)."""
    off = (got.double().view(y.shape) - y).abs() - (2.0 ** -8 * y.abs() + (1 + 2.0 ** -8) * S.F32 * mag + 1e-38)
    assert off.numel() == 0 or off.max().item() <= 0, f"{what}: worst by {off.max().item():.3g}"


def rope_both(rows, hq, hkv, d, rope, pos, n, qn=None, kn=None, in_place=False):
    """lora_qk_rope on [.. Q | K | V ..] rows; results in rows of their own (wider than needed) or in place."""
    s = rows.stride(0)
    k = rows[:, hq * d:(hq + hkv) * d]
    if in_place:
        qo, ko = rows[:, :hq * d], k
    else:
        wide = torch.full((max(n, 1), (hq + hkv) * d + 24), 7.0, dtype=torch.bfloat16, device="cuda")
        qo, ko = wide[:, 8:8 + hq * d], wide[:, 16 + hq * d:16 + (hq + hkv) * d]
    L.lora_qk_rope(rows if hq else None, s, qo if hq else None, qo.stride(0), k if hkv else None, s, ko if hkv else None, ko.stride(0), n, hq, hkv,
                   rope, pos, pos.stride(0), q_norm=qn, k_norm=kn, eps=EPS)
    if not in_place:
        keep = torch.ones_like(wide, dtype=torch.bool)
        keep[:n, 8:8 + hq * d], keep[:n, 16 + hq * d:16 + (hq + hkv) * d] = False, False
        assert (wide[keep] == 7).all()                     # nothing beside the results is written
    return qo[:n], ko[:n]


@pytest.mark.parametrize("d,rot,inter,axes", [(128, 128, False, 1), (128, 128, True, 1), (64, 64, False, 3), (64, 64, True, 2), (128, 48, False, 3),
                                               (128, 8, True, 1), (64, 24, False, 1), (64, 56, True, 4), (128, 120, False, 2), (128, 0, False, 1)])
@pytest.mark.parametrize("n,hq,hkv", [(1, 1, 1), (3, 5, 0), (37, 0, 3), (130, 12, 4), (2100, 28, 4), (9001, 33, 2)])
def test_rows(d, rot, inter, axes, n, hq, hkv):
    g = A.gen(n * 7 + d + rot)
    freqs, axis, rope = rotation(d, rot, axes, inter) if rot else ([], [], L.Rope(d, rotary_dim=0))
    rows = A.randn(g, n, (hq + 2 * hkv) * d + 8, spread=2.0)
    pos = positions(g, axes, n + 3)[:, :n]                 # (rows of positions longer than n)
    norms = [(1 + 0.3 * torch.randn(d, generator=g, device="cuda")).bfloat16() for _ in range(2)]
    for qn, kn in ((None, None), (norms[0], norms[1]), (None, norms[1])):
        q, k = rope_both(rows, hq, hkv, d, rope, pos, n, qn, kn)
        for got, first, heads, norm in ((q, 0, hq, qn), (k, hq, hkv, kn)):
            y, mag = S.turned(rows[:, first * d:(first + heads) * d].double().reshape(n, heads, d), pos, freqs, axis, rot, inter, norm, EPS)
            within(got, y, mag, (qn is not None, heads))


def test_in_place_gives_the_same_bits():
    g = A.gen(3)
    d, n, hq, hkv = 128, 300, 8, 2
    _, _, rope = rotation(d, 64)
    rows, pos = A.randn(g, n, (hq + 2 * hkv) * d), positions(g, 1, n)
    norm = A.randn(g, d)
    q, k = (t.clone() for t in rope_both(rows, hq, hkv, d, rope, pos, n, norm, norm))
    v = rows[:, (hq + hkv) * d:].clone()
    q2, k2 = rope_both(rows, hq, hkv, d, rope, pos, n, norm, norm, in_place=True)
    assert torch.equal(q, q2) and torch.equal(k, k2) and torch.equal(rows[:, (hq + hkv) * d:], v)


def test_far_and_negative_positions():
    """Positions to the ends of int32: the angle is exact to 2^-32 of a turn where float32 has lost all of it. Angles
    here are multiples of 2^-20 turns by construction, so the 64-bit form is exact at every position."""
    d, n = 64, 256
    g = A.gen(5)
    turn = torch.randint(1, 2 ** 20, (32,), generator=g, device="cuda").tolist()
    rope = L.Rope(d)
    for j, t in enumerate(turn):
        rope.struct.turns[j] = t << 44                     # t 2^-20 turns a position
    pos = torch.randint(-2 ** 31, 2 ** 31 - 1, (1, n), generator=g, device="cuda").int()
    pos[0, :4] = torch.tensor([2 ** 31 - 1, -2 ** 31, -1, 2 ** 20], device="cuda", dtype=torch.int32)
    rows = A.randn(g, n, 2 * d)
    out = torch.empty_like(rows)
    L.lora_qk_rope(rows, 2 * d, out, 2 * d, None, 0, None, 0, n, 2, 0, rope, pos, n)
    x = rows.double().view(n, 2, d)
    part = (pos[0].long()[:, None] * torch.tensor(turn, device="cuda")) % 2 ** 20
    a = (part.double() * (2 * torch.pi / 2 ** 20))[:, None]
    x0, x1 = x[..., :32], x[..., 32:]
    y = torch.cat((x0 * a.cos() - x1 * a.sin(), x1 * a.cos() + x0 * a.sin()), -1)
    mag = (x0.abs() + x1.abs()).repeat(1, 1, 2)
    within(out, y, mag, "far")


@pytest.mark.parametrize("d", [64, 128])
def test_values_at_the_edges(d):
    """Rows of zeros, tiny and huge values with a norm (its eps and its f32 sum); NaN and infinities stay in their heads
    and, without a norm, in their pairs."""
    freqs, axis, rope = rotation(d, d)
    x = torch.zeros(8, 2 * d, dtype=torch.float32, device="cuda")
    g = A.gen(9)
    x[1] = 1e-30 * torch.randn(2 * d, generator=g, device="cuda")
    x[2] = 1e15 * torch.randn(2 * d, generator=g, device="cuda")
    x[3:] = torch.randn(5, 2 * d, generator=g, device="cuda")
    x = x.bfloat16()
    pos = positions(g, 1, 8)
    norm = A.randn(g, d)
    q, _ = rope_both(x, 2, 0, d, rope, pos, 8, norm)
    y, mag = S.turned(x.double().view(8, 2, d), pos, freqs, axis, d, False, norm, EPS)
    within(q, y, mag, "edges")
    x[4, 3], x[5, d + 1], x[6, 0] = float("nan"), float("inf"), float("-inf")
    q, _ = rope_both(x, 2, 0, d, rope, pos, 8)
    bad = torch.zeros(8, 2, d, dtype=torch.bool, device="cuda")
    for r, h, e in ((4, 0, 3), (5, 1, 1), (6, 0, 0)):
        bad[r, h, e % (d // 2)] = bad[r, h, e % (d // 2) + d // 2] = True
    got = q.reshape(8, 2, d)
    assert not torch.isfinite(got[bad]).any() and torch.isfinite(got[~bad]).all()
    q, _ = rope_both(x, 2, 0, d, rope, pos, 8, norm)
    bad = torch.zeros(8, 2, dtype=torch.bool, device="cuda")
    bad[4, 0] = True
    assert torch.isnan(q.reshape(8, 2, d)[bad]).all() and torch.isfinite(q.reshape(8, 2, d)[[0, 1, 2, 3, 7]]).all()


def append(rows, hq, hkv, d, rope, pos, n, slots, cache, qn, kn, stream=None, q_out=None):
    s, at = rows.stride(0), rows.data_ptr()
    q = torch.full((max(n, 1), hq * d), 7.0, dtype=torch.bfloat16, device="cuda") if q_out is None else q_out
    L.lora_kv_append(rows if hq else None, s, q if hq else None, q.stride(0), hq, at + 2 * hq * d, s, at + 2 * (hq + hkv) * d, s, slots, n, cache,
                     rope, pos, pos.stride(0), q_norm=qn, k_norm=kn, eps=EPS, stream=stream)
    return q


def fresh(num, kv, page, d, fmt, layout):
    pages = A.pool(num, kv, page, d, fmt, layout, fill=0x5A)
    sc = [None, None] if fmt == "bf16" else [torch.full((num, kv, page), 7.0, device="cuda") for _ in range(2)]
    return pages, sc, L.KvCache(*pages, *sc)


def product_codes(x, fmt):
    """float32 rows [..., D] -> (code values float64, scale float32) by a reciprocal and products, each rounded to float32."""
    q = np.float32(R.QMAX[fmt])
    a = np.abs(x).max(-1)
    y = (x * (q * (np.float32(1) / a))[..., None]).astype(np.float64)
    return R.round_e4m3(y) if fmt == "e4m3" else np.clip(np.rint(y), -127, 127), a * (np.float32(1) / q)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "int8"])
@pytest.mark.parametrize("d,rot,inter,axes,layout", [(128, 128, False, 1, "hnd"), (64, 64, True, 3, "nhd"), (128, 64, False, 2, "kv"), (64, 24, False, 1, "hnd")])
@pytest.mark.parametrize("n,hq,hkv,page", [(1, 2, 1, 1), (3, 0, 2, 7), (37, 8, 4, 16), (515, 9, 3, 64), (4100, 8, 8, 20)])
def test_append(fmt, d, rot, inter, axes, layout, n, hq, hkv, page):
    """q as lora_qk_rope gives it, bit for bit; v by the stated formulas, bit for bit; k within the bounds of one
    rounding to the format; skipped slots and everything else untouched."""
    g = A.gen(n + rot + d)
    freqs, axis, rope = rotation(d, rot, axes, inter)
    num = -(-n // page) + 3
    rows = A.randn(g, n, (hq + 2 * hkv) * d, spread=3.0)
    pos = positions(g, axes, n)
    qn, kn = ((1 + 0.3 * torch.randn(d, generator=g, device="cuda")).bfloat16() for _ in range(2))
    slots = torch.randperm(num * page, generator=g, device="cuda")[:n].clone()
    if n > 2:
        slots[1], slots[2] = -1, num * page
    pages, sc, cache = fresh(num, hkv, page, d, fmt, layout)
    before = rows.clone()
    q = append(rows, hq, hkv, d, rope, pos, n, slots, cache, qn, kn)
    assert torch.equal(rows, before)
    if hq:
        want_q, _ = rope_both(rows, hq, 0, d, rope, pos, n, qn)
        assert torch.equal(q[:n], want_q)
    live = (slots >= 0) & (slots < num * page)
    pg, sl = slots[live] // page, slots[live] % page
    # the slots that were not named
    hit = torch.zeros(num, page, dtype=torch.bool, device="cuda")
    hit[pg, sl] = True
    for x in pages:
        assert ((x.view(torch.uint8) if fmt != "bf16" else x.contiguous().view(torch.uint8)).transpose(1, 2)[~hit] == 0x5A).all()
    for x in sc if fmt != "bf16" else ():
        assert (x.transpose(1, 2)[~hit] == 7).all()
    # v: the formulas, operation by operation
    v = rows[:, (hq + hkv) * d:].reshape(n, hkv, d)[live]
    if fmt == "bf16":
        assert torch.equal(pages[1][pg, :, sl], v)
    else:
        code, scale = product_codes(v.float().cpu().numpy(), fmt)
        assert np.array_equal(pages[1].view(torch.uint8)[pg, :, sl].view(R.DTYPE[fmt]).double().cpu().numpy(), code)
        assert np.array_equal(sc[1][pg, :, sl].cpu().numpy(), scale)
    # k
    y, mag = S.turned(rows[:, hq * d:(hq + hkv) * d].double().reshape(n, hkv, d), pos, freqs, axis, rot, inter, kn, EPS)
    y, mag = y[live], mag[live]
    if fmt == "bf16":
        within(pages[0][pg, :, sl], y, mag, "k")
        return
    scale = sc[0][pg, :, sl].double()[..., None]
    top, e = y.abs().amax(-1, keepdim=True), S.F32 * mag.amax(-1, keepdim=True)
    assert ((scale * R.QMAX[fmt] - top).abs() <= e + 2.0 ** -23 * top).all()
    code = pages[0].view(torch.uint8)[pg, :, sl].view(R.DTYPE[fmt]).double()
    # half a step of the format at the value, its fp32 arithmetic (2 units of 2^-24 of at most the largest), the rotation's error
    half = 0.5 * scale if fmt == "int8" else torch.maximum(2.0 ** -4 * (y.abs() + e), 2.0 ** -10 * scale)
    assert ((code * scale - y).abs() <= half + 2.0 ** -22 * top + 2 * e).all()


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "int8"])
@pytest.mark.parametrize("d,inter,n", [(64, False, 4003), (64, True, 4001), (128, False, 2003)])
def test_append_in_large_calls(fmt, d, inter, n):
    """Heads in fours and tokens side by side in a warp, neither count a multiple."""
    test_append(fmt, d, d, inter, 1, "hnd", n, 33, 4, 16)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_append_rows_that_are_not_finite_or_all_but_zero(fmt):
    """A key head with NaN or an infinity: scale NaN, codes 0; one below 2^-100: zeros; its neighbours as ever."""
    d, n = 64, 6
    g = A.gen(4)
    _, _, rope = rotation(d, 32)
    rows = torch.randn(n, 5 * d, generator=g, device="cuda")            # one q head, two k, two v
    rows[1, d + 3], rows[2, d + 40], rows[3, 3 * d] = float("nan"), float("inf"), float("-inf")
    rows[4, d:2 * d] = 0
    rows[5, d:2 * d] *= 2.0 ** -105
    pages, sc, cache = fresh(2, 2, 4, d, fmt, "hnd")
    append(rows.bfloat16(), 1, 2, d, rope, positions(g, 1, n), n, torch.arange(n, device="cuda"), cache, None, None)
    ks, vs = sc[0].transpose(1, 2).reshape(8, 2)[:n], sc[1].transpose(1, 2).reshape(8, 2)[:n]
    kc = pages[0].view(torch.uint8).transpose(1, 2).reshape(8, 2, d)[:n]
    assert torch.isnan(ks).tolist() == [[False] * 2, [True, False], [True, False], [False] * 2, [False] * 2, [False] * 2]
    assert torch.isnan(vs).tolist() == [[False] * 2] * 3 + [[True, False]] + [[False] * 2] * 2
    assert (kc[1:3, 0] == 0).all() and (kc[4:6, 0] == 0).all() and (ks[4:6, 0] == 0).all() and (ks[:, 1] > 0).all()


def test_other_stream_and_graph():
    """Calls go to the given stream; a captured append and rotation replay with new rows, positions and slots."""
    d, n, hq, hkv, page = 128, 21, 4, 2, 8
    g = A.gen(11)
    _, _, rope = rotation(d, 128)
    rows, pos, slots = A.randn(g, n, (hq + 2 * hkv) * d), positions(g, 1, n), torch.randperm(48, generator=g, device="cuda")[:n].clone()
    pages, sc, cache = fresh(6, hkv, page, d, "int8", "hnd")
    q = torch.zeros(n, hq * d, dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        append(rows, hq, hkv, d, rope, pos, n, slots, cache, None, None, stream=s, q_out=q)
    for seed in (1, 2):
        h = A.gen(seed)
        rows.copy_(A.randn(h, *rows.shape))
        pos.copy_(positions(h, 1, n))
        slots.copy_(torch.randperm(48, generator=h, device="cuda")[:n])
        graph.replay()
        torch.cuda.synchronize()
        pages2, sc2, cache2 = fresh(6, hkv, page, d, "int8", "hnd")
        q2 = append(rows, hq, hkv, d, rope, pos, n, slots, cache2, None, None)
        pg, sl = slots // page, slots % page
        assert torch.equal(q, q2)
        for a, b in ((pages, pages2), (sc, sc2)):
            for j in range(2):
                assert torch.equal(a[j][pg, :, sl], b[j][pg, :, sl])
