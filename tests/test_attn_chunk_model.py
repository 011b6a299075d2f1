"""A CPU model of how lora_attn_chunk shares a batch out (csrc/attn_chunk.cu): key tiles that rows see, cuts of the units,
pieces, the CTAs of an item and the joins' slots. For any lengths every key tile that some row sees is in one piece, the
parts of an item are those of the CTAs that its join counts, no two joins share a slot or a head, and the workspace holds
them."""
from __future__ import annotations

import os
import random
import re

import pytest

SRC = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gather_lora_gb300", "csrc",
                        "attn_chunk.cu")).read()


def const(name):
    return int(re.search(rf"constexpr int {name} = (\d+)[;,]", SRC).group(1))


TILE, MOST, SNAP = const("kTile"), const("kMostCtas"), const("kSnap")
COST, LEAST = const("kItemCost"), const("kLeast")
EVERY = 2 ** 31 - 1


def span(first, end, window, sinks):
    """(low, kept, skip, tiles) of rows at positions first .. end."""
    if end < 0:
        return 0, 0, 0, 0
    low = first - window + 1 if first >= window else 0
    kept = -(-min(sinks, low) // TILE)
    skip = max(0, low // TILE - kept)
    return low, kept, skip, end // TILE + 1 - skip


def items(seqs, step, subs, window, sinks):
    """(sequence, sub, pair, first unit, tiles) in the kernel's order, and the units in all: an item's are its tiles and COST
    before them."""
    out, u = [], 0
    for b, (n, length) in enumerate(seqs):
        np = -(-n // step)
        for sub in range(subs):
            for x in range(np):
                t = span(length - n + x * step, length - n + min((x + 1) * step, n) - 1, window, sinks)[3]
                if t:
                    out.append((b, sub, x, u, t))
                    u += COST + t
    return out, u


def plan(every, total, grid):
    """Pieces of each CTA: (item, first tile, tiles), and the number of CTAs with work."""
    ctas = min(grid, -(-total // LEAST))
    snap = min(SNAP, total // max(ctas, 1) // 4)
    if not ctas:
        return [], 0, snap
    ends = []
    at = 0
    for c in range(ctas + 1):
        r = c * total // ctas
        if r >= total:
            ends.append(total)
            continue
        while every[at][3] + COST + every[at][4] <= r:
            at += 1
        s0, tiles = every[at][3:]
        tile = r - s0 - COST
        ends.append(s0 if tile <= snap else s0 + COST + tiles if tiles - tile <= snap else r)
    pieces = []
    at = 0
    for c in range(ctas):
        mine, u = [], ends[c]
        while u < ends[c + 1]:
            while every[at][3] + COST + every[at][4] <= u:
                at += 1
            s0, tiles = every[at][3:]
            ta = max(0, u - s0 - COST)
            n = min(tiles, ends[c + 1] - s0 - COST) - ta
            mine.append((at, ta, n))
            u = s0 + COST + ta + n
        pieces.append(mine)
    return pieces, ctas, snap


def check(seqs, step, subs, window, sinks, grid):
    every, total = items(seqs, step, subs, window, sinks)
    pieces, ctas, snap = plan(every, total, grid)
    assert ctas <= grid <= MOST
    parts = {}
    for c, mine in enumerate(pieces):
        for at, ta, n in mine:
            assert n > 0
            parts.setdefault(at, []).append((c, ta, n))
    heads, slots = set(), set()
    for at, (b, sub, x, s0, tiles) in enumerate(every):
        got = parts[at]
        assert [ta for _, ta, _ in got] == [sum(n for _, _, n in got[:k]) for k in range(len(got))] and sum(n for _, _, n in got) == tiles
        if len(got) == 1:
            continue
        # the CTAs of the item as the kernel works them out, its slots, and the head that its first CTA writes
        c0 = -(-((s0 + COST + snap + 1) * ctas) // total) - 1
        c1 = -(-((s0 + COST + tiles - snap) * ctas) // total) - 1
        assert [c for c, _, _ in got] == list(range(c0, c1 + 1)), (got, c0, c1)
        for c, ta, _ in got:
            slot = 2 * c + (ta == 0)
            assert (ta == 0) == (c == c0) and slot not in slots and slot < 2 * MOST
            slots.add(slot)
        assert c0 not in heads and c0 < MOST
        heads.add(c0)


@pytest.mark.parametrize("seed", range(150))
def test_every_unit_has_one_cta(seed):
    r = random.Random(seed)
    step = r.choice((2, 4, 16, 32, 42, 64, 128, 256))
    many = r.choice((1, 2, 5, 40))
    seqs = []
    for _ in range(r.randint(1, many)):
        n = r.choice((0, 1, 1, r.randint(1, 20), r.randint(1, 1500)))
        seqs.append((n, r.choice((0, n, n + r.randint(0, 300), r.randint(0, n + 1), n + r.randint(0, 60000)))))
    window, sinks = r.choice((EVERY, r.randint(1, 300), r.randint(1, 9000))), r.choice((0, 4, r.randint(0, 2000), EVERY))
    check(seqs, step, r.choice((1, 2, 4, 8, 16)), window, sinks, r.choice((1, 3, 148, 152, MOST)))


def test_one_item_over_every_cta():
    for n in (TILE * 2 * MOST, TILE * 1000, 2 ** 31 - 64):
        check([(1, n)], 2, 1, EVERY, 0, MOST)
        check([(3, n), (1, 5), (300, n)], 32, 1, EVERY, 0, 152)


@pytest.mark.parametrize("seed", range(60))
def test_tiles_are_those_that_some_row_sees(seed):
    """The tiles numbered without the gap are in order, hold every token that a row sees, and each holds one (or lies
    between the first tokens and the window's, where both meet inside a tile)."""
    r = random.Random(seed)
    n, length = r.randint(1, 300), r.randint(0, 2500)
    first, end = length - n, length - 1
    window, sinks = r.choice((EVERY, r.randint(1, 400), r.randint(1, 2000))), r.choice((0, r.randint(0, 600), EVERY))
    low, kept, skip, tiles = span(first, end, window, sinks)
    at = [t if t < kept else t + skip for t in range(tiles)]
    assert at == sorted(set(at))
    seen = {t for p in range(max(first, 0), end + 1) for t in range(p + 1) if t > p - window or t < sinks}
    assert {t // TILE for t in seen} <= set(at)
    assert seen <= {t for t in range(max(end + 1, 0)) if t >= low or t < sinks}
    if end >= 0:
        assert at[-1] == end // TILE and all(t * TILE < max(sinks, 0) or (t + 1) * TILE > low for t in at)


def test_the_workspace_holds_the_slots():
    head, heads = int(re.search(r"kHead = (\d+)", SRC).group(1)), int(re.search(r"kHeadBytes = (\d+);", SRC).group(1))
    for d in (64, 128):
        slot = 2 * 2 * TILE + 2 * TILE * d + 4
        assert heads + 2 * MOST * slot * 4 <= 48 << 20 and MOST * head <= heads
        assert slot % 4 == 0 and heads % 16 == 0
