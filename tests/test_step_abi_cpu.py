"""lora_rope_init, lora_qk_rope, lora_kv_append, lora_attn_decode_window and lora_attn_chunk on the CPU: refusals on the
host before any CUDA call, no-ops, and the rotation's table. No kernel is launched here."""
from __future__ import annotations

import ctypes
import math
import os
from fractions import Fraction

import pytest
import torch

import step_refs as S
from gather_lora_gb300 import lib as L
from test_attn_abi_cpu import CACHE_FAULTS, FAKE, _cache

NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not os.path.exists(L.LIB_PATH):
        from gather_lora_gb300 import build
        build.build()
    L.load()


def _rope(d=128, **kw):
    r = L.Rope(d).struct
    for k, v in kw.items():
        if k == "axis0":
            r.axis[0] = v
        else:
            setattr(r, k, v)
    return r


ROPE_FAULTS = [(dict(head_dim=96), -2), (dict(rotary_dim=-8), -2), (dict(rotary_dim=136), -2), (dict(rotary_dim=20), -2),
               (dict(axes=0), -2), (dict(axes=5), -2), (dict(axis0=1), -2)]


def _qk(rope=None, **kw):
    a = dict(q=FAKE, qs=1024, qo=FAKE, qos=1024, k=FAKE, ks=512, ko=FAKE, kos=512, n=5, h=8, kv=4, pos=FAKE, ps=5, qn=None, kn=None, eps=1e-6)
    a.update(kw)
    r = _rope() if rope is None else rope
    return L.load().lora_qk_rope(a["q"], a["qs"], a["qo"], a["qos"], a["k"], a["ks"], a["ko"], a["kos"], a["n"], a["h"], a["kv"],
                                 ctypes.byref(r) if r != 0 else None, a["pos"], a["ps"], a["qn"], a["kn"], a["eps"], None)


ROW_FAULTS = [(dict(n=-1), -2), (dict(n=(1 << 24) + 1, ps=1 << 25), -2), (dict(h=-1), -2), (dict(h=1025, qs=1 << 18, qos=1 << 18), -2),
              (dict(qs=1016), -3), (dict(qos=8), -3), (dict(qs=1028), -4), (dict(qos=1025), -4), (dict(ks=504), -3), (dict(ks=516), -4),
              (dict(q=None), -1), (dict(qo=None), -1), (dict(k=None), -1), (dict(pos=None), -1), (dict(ps=4), -3),
              (dict(q=FAKE + 8), -4), (dict(qo=FAKE + 2), -4), (dict(k=FAKE + 4), -4), (dict(qn=FAKE + 8), -4), (dict(kn=FAKE + 2), -4),
              (dict(qn=FAKE, eps=-1.0), -2), (dict(kn=FAKE, eps=NAN), -2), (dict(kn=FAKE, eps=INF), -2)]


def test_qk_rope_refusals():
    for kw, code in ROW_FAULTS + [(dict(kos=504), -3), (dict(kos=520 + 4), -4), (dict(ko=None), -1), (dict(ko=FAKE + 8), -4),
                                  (dict(kv=-1), -2), (dict(kv=1025), -2), (dict(h=0, kv=0), -2)]:
        assert _qk(**kw) == code, kw
        assert L.lora_last_error()
    for kw, code in ROPE_FAULTS:
        assert _qk(rope=_rope(**kw)) == code, kw
    assert _qk(rope=0) == -1
    assert _qk(n=0, q=None, qo=None, k=None, ko=None, pos=None) == 0
    assert L.lora_last_error() == ""


def _append(rope=None, cache=None, **kw):
    a = dict(q=FAKE, qs=1024, qo=FAKE, qos=1024, h=8, k=FAKE, ks=512, v=FAKE, vs=512, slots=FAKE, n=5, pos=FAKE, ps=5, qn=None, kn=None, eps=1e-6)
    a.update(kw)
    r = _rope() if rope is None else rope
    c = _cache() if cache is None else cache
    return L.load().lora_kv_append(a["q"], a["qs"], a["qo"], a["qos"], a["h"], a["k"], a["ks"], a["v"], a["vs"], a["slots"], a["n"],
                                   ctypes.byref(c) if c != 0 else None, ctypes.byref(r) if r != 0 else None, a["pos"], a["ps"],
                                   a["qn"], a["kn"], a["eps"], None)


def test_kv_append_refusals():
    for kw, code in ROW_FAULTS + [(dict(vs=504), -3), (dict(vs=516), -4), (dict(v=None), -1), (dict(v=FAKE + 8), -4), (dict(slots=None), -1)]:
        assert _append(**kw) == code, kw
        assert L.lora_last_error()
    for kw, code in CACHE_FAULTS:
        assert _append(cache=_cache(**kw)) == code, kw
    for kw, code in ROPE_FAULTS:
        assert _append(rope=_rope(**kw)) == code, kw
    assert _append(rope=0) == -1 and _append(cache=0) == -1
    assert _append(rope=_rope(64)) == -2                   # a rotation of another head size than the cache's
    assert _append(n=0, q=None, qo=None, k=None, v=None, slots=None, pos=None) == 0


def _window(fn, cache=None, **kw):
    a = dict(q=FAKE, qs=1024, out=FAKE, os=1024, cu=FAKE, b=4, tq=9, h=8, scale=0.1, table=FAKE, ts=32, mp=32, lens=FAKE, w=100, s=4,
             lse=None, ws=FAKE, wb=L.CHUNK_WORKSPACE if fn == "lora_attn_chunk" else L.ATTN_WORKSPACE)
    a.update(kw)
    c = _cache() if cache is None else cache
    chunk = (a["cu"], a["b"], a["tq"]) if fn == "lora_attn_chunk" else (a["b"],)
    return getattr(L.load(), fn)(a["q"], a["qs"], a["out"], a["os"], *chunk, a["h"], a["scale"], ctypes.byref(c) if c != 0 else None,
                                 a["table"], a["ts"], a["mp"], a["lens"], a["w"], a["s"], a["lse"], a["ws"], a["wb"], None)


@pytest.mark.parametrize("fn", ["lora_attn_decode_window", "lora_attn_chunk"])
def test_window_and_chunk_refusals(fn):
    faults = [(dict(b=-1), -2), (dict(b=8193), -2), (dict(h=0), -2), (dict(h=6), -2), (dict(h=1028), -2), (dict(scale=0.0), -2),
              (dict(scale=-1.0), -2), (dict(scale=NAN), -2), (dict(scale=INF), -2), (dict(mp=-1), -2), (dict(mp=1 << 28, ts=1 << 28), -2),
              (dict(qs=1016), -3), (dict(os=8), -3), (dict(qs=1028), -4), (dict(os=1025), -4), (dict(ts=31), -3), (dict(q=None), -1),
              (dict(out=None), -1), (dict(lens=None), -1), (dict(ws=None), -1), (dict(table=None), -1), (dict(q=FAKE + 2), -4),
              (dict(out=FAKE + 8), -4), (dict(ws=FAKE + 4), -4), (dict(w=0), -2), (dict(w=-5), -2), (dict(s=-1), -2)]
    if fn == "lora_attn_chunk":
        faults += [(dict(tq=-1), -2), (dict(tq=(1 << 24) + 1), -2), (dict(cu=None), -1), (dict(wb=L.CHUNK_WORKSPACE - 1), -2)]
        assert _window(fn, tq=0, q=None, out=None, cu=None) == 0
    else:
        faults += [(dict(wb=L.ATTN_WORKSPACE - 1), -2)]
    for kw, code in faults:
        assert _window(fn, **kw) == code, kw
        assert L.lora_last_error()
    for kw, code in CACHE_FAULTS:
        assert _window(fn, cache=_cache(**kw)) == code, kw
    assert _window(fn, cache=0) == -1
    assert _window(fn, b=0, q=None, out=None, lens=None, ws=None, table=None, cu=None) == 0


def test_rope_init_refusals():
    def init(d=128, rot=8, freqs=(1.0, 0.1, 0.01, 0.001), axis=None, axes=1, rope=True):
        r = L._RopeStruct()
        r.axes = 77
        rc = L.load().lora_rope_init(ctypes.byref(r) if rope else None, d, rot, (ctypes.c_double * 4)(*freqs) if freqs else None,
                                     (ctypes.c_uint8 * 4)(*axis) if axis else None, axes, 0)
        assert rc == 0 or r.axes == 77                     # nothing is written by a refused call
        return rc
    assert init() == 0 and init(axis=(0, 2, 1, 0), axes=3) == 0 and init(rot=0, freqs=None) == 0
    for kw, code in [(dict(rope=False), -1), (dict(d=80), -2), (dict(rot=12), -2), (dict(rot=-8), -2), (dict(rot=136), -2), (dict(freqs=None), -1),
                     (dict(axes=0), -2), (dict(axes=5), -2), (dict(axis=(0, 1, 0, 0)), -2), (dict(freqs=(1.0, NAN, 1.0, 1.0)), -2),
                     (dict(freqs=(1.0, 1.0, 1.0, INF)), -2)]:
        assert init(**kw) == code, kw


def test_rope_object_checks_its_arguments():
    r = L.Rope(128, rotary_dim=48, sections=(4, 10, 10)).struct
    assert (r.head_dim, r.rotary_dim, r.axes, r.interleaved) == (128, 48, 3, 0)
    assert list(r.axis[:24]) == [0] * 4 + [1] * 10 + [2] * 10
    assert L.Rope(64, axis=[j % 2 for j in range(32)], interleaved=True).struct.axes == 2
    for kw in (dict(sections=(30, 30)), dict(freqs=[1.0] * 63), dict(axis=[0] * 10), dict(sections=(64,), axis=[0] * 64), dict(axis=[300] * 64),
               dict(sections=(70, -6))):
        with pytest.raises(ValueError):
            L.Rope(128, **kw)
    for kw in (dict(rotary_dim=20), dict(rotary_dim=136), dict(axis=[5] * 64)):
        with pytest.raises(L.LoraError):
            L.Rope(128, **kw)
    with pytest.raises(L.LoraError):
        L.Rope(96)


def test_table_holds_the_turns():
    """turns[j] is freqs[j] / (2 pi) less its whole part, in units of 2^-64: off by 2^-62 and by what the two roundings to
    double leave (2^-52 of the quotient, whole part included); positions then wrap around exactly."""
    # pi to 60 digits
    pi = Fraction(314159265358979323846264338327950288419716939937510582097494, 10 ** 59)
    freqs = [1.0, 0.5, 10000.0 ** -0.75, 1e-9, 0.0, 6.283185307179586, 1234.5, -0.3, -1e-22, 3e5, 0.1, 2.0 ** -40]
    r = L.Rope(128, rotary_dim=24, freqs=freqs).struct
    for f, t in zip(freqs, r.turns):
        want = Fraction(f) / (2 * pi)
        off = (Fraction(int(t), 2 ** 64) - want) % 1
        off = min(off, 1 - off)
        assert off <= Fraction(1, 2 ** 62) + abs(want) * Fraction(1, 2 ** 52), f


def test_reference_rotation_and_window():
    """The references against closed forms: rotating by p then by -p is nothing, angles add, and the window's mask."""
    g = torch.Generator().manual_seed(1)
    x = torch.randn(7, 2, 64, generator=g, dtype=torch.float64)
    pos = torch.tensor([[0, 1, 5, 100, -3, 17, 2 ** 20]])
    freqs = [10000.0 ** (-2 * j / 64) for j in range(32)]
    for inter in (False, True):
        y, _ = S.turned(x, pos, freqs, [0] * 32, 64, inter)
        back, _ = S.turned(y, -pos, freqs, [0] * 32, 64, inter)
        assert torch.allclose(back, x, atol=1e-12) and torch.allclose(y[0], x[0])
        assert torch.allclose(y.norm(dim=-1), x.norm(dim=-1))
    m = S.seen(3, 6, 2, 1, device="cpu")
    assert m.int().tolist() == [[1, 0, 1, 1, 0, 0], [1, 0, 0, 1, 1, 0], [1, 0, 0, 0, 1, 1]]
    assert S.seen(4, 2, 100, 0, device="cpu").int().tolist() == [[0, 0], [0, 0], [1, 0], [1, 1]]
    y, _ = S.turned(x, pos, freqs[:4], [0] * 4, 8, False, norm=torch.ones(64), eps=0.0)
    assert torch.allclose(y.square().mean(-1), torch.ones(7, 2, dtype=torch.float64))
    assert math.isclose(S.F32, 2.0 ** -18)
