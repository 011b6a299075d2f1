"""The cache and attention calls on the CPU: refusals on the host before any CUDA call, no-ops,
and the 64-bit reference's rounding. No kernel is launched here."""
from __future__ import annotations

import ctypes
import os

import numpy as np
import pytest
import torch

import attn_refs as R
from gather_lora_gb300 import lib as L

FAKE = 0x100000            # a non-NULL, 16-byte aligned address that is never dereferenced


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not os.path.exists(L.LIB_PATH):
        from gather_lora_gb300 import build
        build.build()
    L.load()


def _cache(**kw):
    a = dict(k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, ps=16 * 4 * 128, hs=16 * 128, ts=128, pages=64, heads=4, page=16, d=128,
             fmt=L.KV_INT8)
    a.update(kw)
    return L._KvCacheStruct(a["k"], a["v"], a["ks"], a["vs"], a["ps"], a["hs"], a["ts"], a["pages"], a["heads"],
                            a["page"], a["d"], a["fmt"])


CACHE_FAULTS = [
    (dict(fmt=-1), -2), (dict(fmt=3), -2), (dict(d=96), -2), (dict(d=0), -2), (dict(heads=0), -2), (dict(heads=1025), -2),
    (dict(pages=-1), -2), (dict(page=0), -2), (dict(k=None), -1), (dict(v=None), -1), (dict(ks=None), -1), (dict(vs=None), -1),
    (dict(k=FAKE + 8), -4), (dict(v=FAKE + 2), -4), (dict(ks=FAKE + 2), -4), (dict(ps=16 * 4 * 128 + 8), -4),
    (dict(hs=100), -4), (dict(ts=120), -4), (dict(ts=112), -3), (dict(ps=64), -3), (dict(hs=-128), -3),
    (dict(fmt=0, ts=132), -4),
]


def _rows(fn, cache=None, **kw):
    a = dict(k=FAKE, ks=512, v=FAKE, vs=512, slots=FAKE, n=5)
    a.update(kw)
    c = _cache() if cache is None else cache
    return getattr(L.load(), fn)(a["k"], a["ks"], a["v"], a["vs"], a["slots"], a["n"],
                                 ctypes.byref(c) if c != 0 else None, None)


@pytest.mark.parametrize("fn", ["lora_kv_write", "lora_kv_read"])
def test_kv_rows_refusals(fn):
    for kw, code in [(dict(n=-1), -2), (dict(n=(1 << 24) + 1), -2), (dict(ks=504), -3), (dict(vs=8), -3),
                     (dict(ks=516), -4), (dict(vs=513), -4), (dict(k=None), -1), (dict(v=None), -1),
                     (dict(slots=None), -1), (dict(k=FAKE + 2), -4), (dict(v=FAKE + 8), -4)]:
        assert _rows(fn, **kw) == code, kw
        assert L.lora_last_error()
    for kw, code in CACHE_FAULTS:
        assert _rows(fn, cache=_cache(**kw)) == code, kw
    assert _rows(fn, cache=0) == -1
    assert _rows(fn, n=0, k=None, v=None, slots=None) == 0
    assert L.lora_last_error() == ""


def _decode(cache=None, **kw):
    a = dict(q=FAKE, qs=1024, out=FAKE, os=1024, b=4, h=8, scale=0.1, table=FAKE, ts=32, mp=32, lens=FAKE, lse=None,
             ws=FAKE, wb=L.ATTN_WORKSPACE)
    a.update(kw)
    c = _cache() if cache is None else cache
    return L.load().lora_attn_decode(a["q"], a["qs"], a["out"], a["os"], a["b"], a["h"], a["scale"],
                                     ctypes.byref(c) if c != 0 else None, a["table"], a["ts"], a["mp"], a["lens"],
                                     a["lse"], a["ws"], a["wb"], None)


def test_decode_refusals():
    for kw, code in [(dict(b=-1), -2), (dict(b=8193), -2), (dict(h=0), -2), (dict(h=6), -2), (dict(h=1028), -2),
                     (dict(scale=0.0), -2), (dict(scale=-1.0), -2), (dict(scale=float("nan")), -2),
                     (dict(scale=float("inf")), -2), (dict(mp=-1), -2), (dict(mp=1 << 28, ts=1 << 28), -2),
                     (dict(qs=1016), -3), (dict(os=8), -3), (dict(qs=1028), -4), (dict(os=1025), -4), (dict(ts=31), -3),
                     (dict(wb=L.ATTN_WORKSPACE - 1), -2), (dict(q=None), -1), (dict(out=None), -1), (dict(lens=None), -1),
                     (dict(ws=None), -1), (dict(table=None), -1), (dict(q=FAKE + 2), -4), (dict(out=FAKE + 8), -4),
                     (dict(ws=FAKE + 4), -4)]:
        assert _decode(**kw) == code, kw
        assert L.lora_last_error()
    for kw, code in CACHE_FAULTS:
        assert _decode(cache=_cache(**kw)) == code, kw
    assert _decode(cache=0) == -1
    # the longest sequence a table may describe: 2^31 - 64 tokens
    assert _decode(cache=_cache(page=2 ** 30 - 32, pages=1), mp=2, ts=2, q=None) == -1      # allowed: on to the next check
    assert _decode(cache=_cache(page=2 ** 31 - 63, pages=1), mp=1, ts=1, q=None) == -2
    assert _decode(b=0, q=None, out=None, lens=None, ws=None, table=None) == 0


def _prefill(**kw):
    a = dict(q=FAKE, qs=1024, k=FAKE, ks=512, v=FAKE, vs=512, out=FAKE, os=1024, cq=FAKE, ck=FAKE, b=2, tq=100, tk=200,
             h=8, kv=4, d=128, scale=0.1, lse=None)
    a.update(kw)
    return L.load().lora_attn_prefill(a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["out"], a["os"], a["cq"],
                                      a["ck"], a["b"], a["tq"], a["tk"], a["h"], a["kv"], a["d"], a["scale"], a["lse"],
                                      None)


def test_prefill_refusals():
    for kw, code in [(dict(b=-1), -2), (dict(b=8193), -2), (dict(tq=-1), -2), (dict(tk=-1), -2),
                     (dict(tq=(1 << 24) + 1), -2), (dict(tk=(1 << 24) + 1), -2), (dict(d=80), -2), (dict(kv=0), -2),
                     (dict(h=9), -2), (dict(h=2048), -2), (dict(scale=0.0), -2), (dict(scale=float("nan")), -2),
                     (dict(qs=1000), -3), (dict(ks=504), -3), (dict(vs=504), -3), (dict(os=1016), -3), (dict(qs=1028), -4),
                     (dict(ks=514), -4), (dict(vs=516), -4), (dict(os=1030), -4), (dict(q=None), -1), (dict(k=None), -1),
                     (dict(v=None), -1), (dict(out=None), -1), (dict(cq=None), -1), (dict(ck=None), -1),
                     (dict(q=FAKE + 2), -4), (dict(k=FAKE + 8), -4), (dict(v=FAKE + 4), -4), (dict(out=FAKE + 2), -4)]:
        assert _prefill(**kw) == code, kw
        assert L.lora_last_error()
    assert _prefill(b=0, q=None) == 0
    assert _prefill(tq=0, q=None, k=None) == 0


def test_cache_object_checks_its_tensors():
    def t(*shape, dtype=torch.int8):
        return torch.zeros(shape, dtype=dtype)
    pages, scale = t(3, 2, 4, 64), torch.zeros(3, 2, 4)
    c = L.KvCache(pages, pages.clone(), scale, scale.clone())
    assert (c.struct.num_pages, c.struct.kv_heads, c.struct.page_size, c.struct.head_dim, c.struct.format) == (3, 2, 4, 64, L.KV_INT8)
    assert (c.struct.page_stride, c.struct.head_stride, c.struct.token_stride) == (512, 256, 64)
    nhd = t(3, 4, 2, 64).transpose(1, 2)      # [page, slot, head, d] storage
    c = L.KvCache(nhd, nhd, scale, scale)
    assert (c.struct.head_stride, c.struct.token_stride) == (64, 128)
    for bad in [(pages, pages.bfloat16()), (pages.half(), pages.half()), (pages, t(3, 2, 5, 64), scale, scale),
                (pages, nhd, scale, scale), (pages, pages), (pages, pages, scale.double(), scale),
                (pages, pages, scale, torch.zeros(3, 4, 2).transpose(1, 2)), (t(3, 2, 64), t(3, 2, 64))]:
        with pytest.raises(ValueError):
            L.KvCache(*bad)


def test_reference_rounding_is_the_formats():
    """Every E4M3 code is a fixed point of the reference's rounding, and midpoints go to even."""
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    vals = np.unique(codes[np.isfinite(codes)])
    assert len(vals) == 253 and np.array_equal(R.round_e4m3(vals), vals)
    mid = (vals[1:] + vals[:-1]) / 2
    want = torch.from_numpy(mid).float().to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(R.round_e4m3(mid), want)
    assert R.round_e4m3(np.array([500.0, -1e9])).tolist() == [448.0, -448.0]


def test_reference_attention_is_softmax():
    g = torch.Generator().manual_seed(0)
    q, k, v = (torch.randn(s, 64, generator=g, dtype=torch.float64) for s in (5, 9, 9))
    seen = torch.arange(9) <= torch.arange(5)[:, None] + 2
    out, lse, _ = R.attend(q, k, v, 0.3, seen)
    z = (0.3 * q @ k.T).masked_fill(~seen, -torch.inf)
    assert torch.allclose(out, torch.softmax(z, 1) @ v, atol=1e-13) and torch.allclose(lse, torch.logsumexp(z, 1))
    none, l0, _ = R.attend(q, k, v, 0.3, torch.zeros(5, 9, dtype=torch.bool))
    assert (none == 0).all() and torch.isinf(l0).all()
