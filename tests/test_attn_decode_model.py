"""A CPU model of how lora_attn_decode deals a batch's tiles to CTAs and joins the parts: the kernel's
index arithmetic restated step by step, its constants read from the source. Whatever the lengths, every
tile belongs to one CTA, no two parts share a workspace slot, no two joins share a counter, and each
counter sees exactly the arrivals it waits for."""
from __future__ import annotations

import bisect
import os
import random
import re

import pytest

SRC = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gather_lora_gb300", "csrc",
                        "attn_decode.cu")).read()


def const(name):
    return int(re.search(rf"constexpr int {name} = (\d+);", SRC).group(1))


WARPS, GROUP, MAX_CTAS, PER_SM = const("kDecWarps"), const("kJoinGroup"), const("kMaxCtas"), const("kCtasPerSm")
WHOLE = int(re.search(r"constexpr int kWhole = (\d+) \* kDecWarps;", SRC).group(1)) * WARPS


def plan(tiles, subs, grid, shared_counters=False):
    """tiles: per sequence. Returns the parts of each segment as (cta, slot, counter) lists after checking them."""
    total = sum(tiles) * subs
    if total == 0:
        return {}
    n = min(grid, (total + WARPS - 1) // WARPS)
    segments, at = [], 0
    for t in tiles:
        for _ in range(subs if t else 0):
            segments.append((at, t))
            at += t
    covered, parts, i0 = 0, {}, 0

    def end(u):
        """An equal share's end, moved to the nearer end of a segment of at most WHOLE tiles."""
        s0, t = segments[bisect.bisect_right(starts, u) - 1] if u < total else (total, 0)
        return u if t > WHOLE or u == total else (s0 if 2 * (u - s0) < t else s0 + t)
    starts = [s0 for s0, _ in segments]
    for c in range(n):
        u0, u1 = end(c * total // n), end((c + 1) * total // n)
        assert u0 == covered and u1 >= u0
        covered = u1
        u, i = u0, i0
        while u < u1:
            while segments[i][0] + segments[i][1] <= u:
                i += 1
            s0, t = segments[i]
            ta = u - s0
            tb = min(t, ta + (u1 - u))
            if not (ta == 0 and tb == t):
                assert t > WHOLE
                parts.setdefault((s0, t), []).append((c, 2 * c + (ta == 0)))
            u += tb - ta
        i0 = i
    assert covered == total
    slots, counters = set(), {}
    for (s0, t), got in parts.items():
        c0, c1 = ((s0 + 1) * n - 1) // total, ((s0 + t) * n - 1) // total
        assert [c for c, _ in got] == list(range(c0, c1 + 1))
        for c, slot in got:
            assert slot == 2 * c + (c == c0) and slot not in slots and slot < 2 * MAX_CTAS
            slots.add(slot)
            gi = (c - c0) // GROUP
            first = c0 + gi * GROUP
            key = (MAX_CTAS if gi and not shared_counters else 0) + first
            want = min(GROUP, c1 - first + 1)
            owner = counters.setdefault(key, [(s0, t), want, 0])
            assert owner[0] == (s0, t), "two segments at one counter"
            owner[2] += 1
        groups = (c1 - c0) // GROUP + 1
        if groups > 1:
            assert 2 * MAX_CTAS + c0 not in counters
            counters[2 * MAX_CTAS + c0] = [(s0, t), groups, groups]
    assert all(seen == want for _, want, seen in counters.values()) and all(k < 3 * MAX_CTAS for k in counters)
    return parts


@pytest.mark.parametrize("seed", range(40))
def test_any_lengths(seed):
    r = random.Random(seed)
    tiles = [r.choice((0, 1, 2, 3, r.randrange(1, 40), r.randrange(1, 4000))) for _ in range(r.choice((1, 2, 5, 40, 300)))]
    plan(tiles, r.choice((1, 2, 3, 8, 24)), r.choice((1, 2, 7, 152 * PER_SM, MAX_CTAS)))


@pytest.mark.parametrize("tiles,subs", [([1], 1), ([6251], 2), ([1], 1000), ([313, 3, 0, 57], 4), ([0, 0, 0], 8), ([2 ** 27], 4),
                                        ([1, 1, 63, 63, 63, 4, 4, 5, 126, 126, 17], 2)])
def test_chosen_lengths(tiles, subs):
    plan(tiles, subs, 152 * PER_SM)


def test_the_model_sees_a_shared_counter():
    """A segment's last group may start in the CTA where the next segment starts: one counter for both is
    the mistake the separate ones are there for."""
    with pytest.raises(AssertionError, match="two segments at one counter"):
        plan([65, 9, 12], 4, 152 * PER_SM, shared_counters=True)
