"""A CPU model of the joins of lora_attn_decode: how many parts each of them gets, against what the kernel's
shared arrays hold (read from the source), and the joins' arithmetic in 64 bits over random parts. The split
itself is tests/test_attn_decode_model.py's."""
from __future__ import annotations

import random
import re

import numpy as np
import pytest

import test_attn_decode_model as M

NAMES = {"kJoinGroup": M.GROUP, "kMaxCtas": M.MAX_CTAS}
for _name, _a, _b in re.findall(r"constexpr int (\w+) = (\w+) / (\w+);", M.SRC):
    if _a in NAMES and _b in NAMES:
        NAMES[_name] = NAMES[_a] // NAMES[_b]


def held():
    """Parts that the arrays of joined maxima and sums hold."""
    sizes = [NAMES[n] for n in re.findall(r"s_j[ml]\[(\w+) \* kRows\]", re.search(r"__shared__ float s_jm.*", M.SRC).group())]
    assert len(sizes) == 2
    return min(sizes)


def joins(parts):
    """(parts of the join, whether it is a group's) for every join of a plan."""
    for got in parts.values():
        c0, c1 = got[0][0], got[-1][0]
        groups = (c1 - c0) // M.GROUP + 1
        for gi in range(groups):
            yield min(M.GROUP, c1 - (c0 + gi * M.GROUP) + 1), True
        if groups > 1:
            yield groups, False


GRIDS = (1, 2, 17, 152 * M.PER_SM, M.MAX_CTAS)


@pytest.mark.parametrize("grid", GRIDS)
def test_every_join_fits(grid):
    """One long sequence alone or in a batch, one head or several: no join has more parts than the arrays hold."""
    r = random.Random(grid)
    most = 0
    for tiles, subs in ([([n], s) for n in (1, 40, 1025, 2048, 100003, 2 ** 27) for s in (1, 2, 8)] +
                        [([6250, 125, 188], 1), ([0, 1300, 2], 1), ([9] * 100, 1)] +
                        [([r.randrange(1, 4000) for _ in range(r.randrange(1, 4))], r.choice((1, 2))) for _ in range(60)]):
        for count, group in joins(M.plan(tiles, subs, grid)):
            assert count <= (M.GROUP if group else held()), (tiles, subs, grid, count)
            most = max(most, count if not group else 0)
    assert most == (-(-grid // M.GROUP) if grid > M.GROUP else 0)      # the sweep reaches a segment over the whole grid


def test_grids_are_bounded():
    """The launcher gives at most kMaxCtas CTAs, and that many make no more groups than a join holds."""
    assert re.search(r"sms \* kCtasPerSm < kMaxCtas \? sms \* kCtasPerSm : kMaxCtas", M.SRC)
    assert -(-M.MAX_CTAS // M.GROUP) <= held()


def join(m, l, o, rounds=None):
    """Parts joined as the kernel does: all maxima first, then sums in rounds of GROUP parts."""
    mm = m.max()
    ref = 0.0 if mm == -np.inf else mm
    ll, acc = 0.0, np.zeros(o.shape[1])
    for x0 in list(range(0, len(m), M.GROUP))[:rounds]:
        for x in range(x0, min(x0 + M.GROUP, len(m))):
            f = np.exp2(m[x] - ref)
            ll, acc = ll + l[x] * f, acc + o[x] * f
    return mm, ll, acc


def two_levels(m, l, o, rounds=None):
    got = [join(m[i:i + M.GROUP], l[i:i + M.GROUP], o[i:i + M.GROUP]) for i in range(0, len(m), M.GROUP)]
    mm, ll, acc = join(np.array([g[0] for g in got]), np.array([g[1] for g in got]), np.array([g[2] for g in got]), rounds)
    return mm + np.log2(ll), acc / ll


def parts(count, seed):
    g = np.random.default_rng(seed)
    z, v = g.normal(size=(count, 50)) * 3, g.normal(size=(count, 50, 8))
    z[count // 2] = -np.inf                       # a part that saw no token
    m = z.max(1)
    w = np.exp2(z - np.where(m == -np.inf, 0.0, m)[:, None])
    return z, v, m, w.sum(1), np.einsum("pt,ptd->pd", w, v)


@pytest.mark.parametrize("count", [2, 16, 17, 256, 257, 303, 304, 512])
def test_the_joins_are_the_softmax(count):
    z, v, m, l, o = parts(count, count)
    w = np.exp2(z - z.max())
    lse, out = two_levels(m, l, o)
    assert abs(lse - (z.max() + np.log2(w.sum()))) < 1e-12
    assert np.abs(out - np.einsum("pt,ptd->d", w, v) / w.sum()).max() < 1e-12


def test_the_model_sees_a_dropped_round():
    """A second level that takes one round of parts alone is far off."""
    z, v, m, l, o = parts(304, 1)
    whole, cut = two_levels(m, l, o), two_levels(m, l, o, rounds=1)
    assert abs(whole[0] - cut[0]) > 0.1
