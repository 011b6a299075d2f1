"""A CPU model of how many CTAs lora_attn_decode_window takes for short windows (csrc/attn_decode.cu): in a batch of equal
lengths, idle sequences among them, no segment has more parts than one join takes."""
from __future__ import annotations

import os
import random
import re

import pytest

SRC = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gather_lora_gb300", "csrc",
                        "attn_decode.cu")).read()
WARPS, GROUP = (int(re.search(rf"constexpr int {name} = (\d+);", SRC).group(1)) for name in ("kDecWarps", "kJoinGroup"))
GRID = 304


def limit(tok):
    """Tiles a segment, of the mean, up to which the rule holds."""
    few, many = re.search(r"constexpr int kMostTokens = \(TOK == 16 \? (\d+) : (\d+)\) \* kDecWarps \* \(kJoinGroup - 1\);", SRC).groups()
    return int(few if tok == 16 else many) * WARPS * (GROUP - 1) // tok


def ctas(tiles, subs, tok, idle_too=False):
    total, segments = sum(tiles) * subs, sum(1 for t in tiles if t or idle_too) * subs
    n = min(GRID, -(-total // WARPS))
    return min(n, (GROUP - 1) * segments) if total <= limit(tok) * segments else n


def parts(tiles, subs, n):
    """CTAs that equal shares of n CTAs give a segment, at most."""
    total, at, worst = sum(tiles) * subs, 0, 0
    for t in tiles:
        for _ in range(subs if t else 0):
            worst = max(worst, ((at + t) * n - 1) // total - ((at + 1) * n - 1) // total + 1)
            at += t
    return worst


@pytest.mark.parametrize("tok", [16, 32, 64])
def test_one_join(tok):
    r = random.Random(tok)
    for _ in range(400):
        most = r.randint(1, limit(tok))
        tiles = [most] * r.randint(1, 5) + [0] * r.choice((0, 1, 7, 100))
        r.shuffle(tiles)
        subs = r.choice((1, 2, 4, 8, 24))
        n = ctas(tiles, subs, tok)
        assert n >= 1 and parts(tiles, subs, n) <= GROUP


def test_counting_idle_sequences_would_join_twice():
    assert parts([128, 0], 4, ctas([128, 0], 4, 16, idle_too=True)) > GROUP


def test_the_kernel_counts_sequences_with_tiles():
    assert "mine += t ? kOneLive : 0" in SRC and "total / kOneLive * subs" in SRC
    assert re.search(r"if \(total <= kMostTokens / TOK \* segments\) n = min\(n, \(kJoinGroup - 1\) \* segments\);", SRC)
