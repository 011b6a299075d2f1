"""A CPU model of the prefill attention's barriers: the TMA, MMA, softmax and look roles of one CTA restated step by
step (csrc/attn_prefill.cu, one step per barrier operation), loads and MMAs that complete later, run in random
order. A wait knows which phase it means: passing on another one's parity, reading a stage, a job or an item slot that holds
something else, or a run that stops short is a failure."""
from __future__ import annotations

import os
import random
import re
from collections import deque

import pytest

SRC = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gather_lora_gb300", "csrc",
                        "attn_prefill.cu")).read()


def const(name):
    return int(re.search(rf"constexpr int (?:\w+ = \d+, )*{name} = (\d+)[;,]", SRC).group(1))


ITEMS, JOBS, LOOKS = const("kItems"), const("kJobs"), const("kScanWarps")
STAGES = {128: int(re.search(r"stages = D == 128 \? (\d+) : \d+", SRC).group(1)),
          64: int(re.search(r"stages = D == 128 \? \d+ : (\d+)", SRC).group(1))}


class Bar:
    """An mbarrier: arrivals and bytes still due in this phase, phases completed."""

    def __init__(self, count):
        self.count = self.due = count
        self.tx = self.phase = 0

    def _turn(self):
        assert self.due >= 0, "more arrivals than a phase has"
        if self.due == 0 and self.tx == 0:
            self.due, self.phase = self.count, self.phase + 1

    def arrive(self, tx=0):
        self.due -= 1
        self.tx += tx
        self._turn()

    def bytes(self, n):
        self.tx -= n
        self._turn()


def wait(bar, k):
    """Until phase k (0, 1, ..) of `bar` is complete, by its parity as the hardware does."""
    while bar.phase & 1 == k & 1:
        yield
    assert bar.phase == k + 1, f"a wait for phase {k} passed in phase {bar.phase}"


def run(items, D, seed, unannounced=False, JOBS=JOBS):
    """items: (n0, n1, whole key tiles) of each."""
    r = random.Random(seed)
    NS, bufs = STAGES[D], 2 if D == 128 else 3
    full, empty = [Bar(1 + (s & 1)) for s in range(NS)], [Bar(1) for _ in range(NS)]
    item_full, item_empty = [Bar(1) for _ in range(ITEMS)], [Bar(2 + 1) for _ in range(ITEMS)]   # (a warpgroup as one actor)
    landed = [Bar(1) for _ in range(JOBS)]
    q_full, q_empty = Bar(1), Bar(1)
    s_full, p_ready, o_done = ([[Bar(1) for _ in range(2)] for _ in range(2)] for _ in range(3))
    slot, job, stage = [None] * (2 * ITEMS), [None] * JOBS, [None] * NS
    looked, stored, bad = {}, [0, 0], {it for it in range(len(items)) if r.random() < 0.3}
    later, pipe = [], deque()            # loads under way; MMAs and commits in order

    def load(bar, s, tile):
        bar.arrive(tx=1)

        def land():
            stage[s] = tile
            looked[tile] = 0
            bar.bytes(1)
        later.append(land)

    def tma():
        kv = jobs = nq = 0
        for it in range(len(items) + 1):
            if it >= ITEMS:
                yield from wait(item_empty[it % ITEMS], it // ITEMS - 1)
            slot[it % (2 * ITEMS)] = it
            item_full[it % ITEMS].arrive()
            yield
            if it == len(items):
                break
            n0, n1, whole = items[it]
            n = max(n0, n1)
            if n == 0:
                continue
            if nq:
                yield from wait(q_empty, nq - 1)
            nq += 1
            load_q = q_full
            load_q.arrive(tx=1)
            later.append(lambda: load_q.bytes(1))
            for j in range(2 * n):
                s = kv % NS
                if kv >= NS:
                    yield from wait(empty[s], kv // NS - 1)
                look = j & 1 and (j >> 1) >= whole
                if look:
                    bar = landed[jobs % JOBS]
                    job[jobs % JOBS] = (it, s, j == 2 * n - 1, kv)
                    jobs += 1
                else:
                    bar = full[s]
                    if j & 1:
                        bar.arrive()
                load(bar, s, kv)
                kv += 1
                yield
        job[jobs % JOBS] = (-1, 0, True, 0)
        landed[jobs % JOBS].arrive()

    def look():
        k, seen = 0, {}
        while True:
            if unannounced:                  # (planted) takes a job as soon as it is written
                while job[k % JOBS] == seen.get(k % JOBS):
                    yield
                seen[k % JOBS] = job[k % JOBS]
            else:
                yield from wait(landed[k % JOBS], k // JOBS)
            it, s, last, tile = job[k % JOBS]
            k += 1
            if it < 0:
                return
            assert stage[s] == tile, "another tile in the stage"
            yield
            assert stage[s] == tile
            looked[tile] += 1
            add = last and it in bad
            if add:
                assert slot[it % (2 * ITEMS)] == it, "the item's slot was used again"
            full[s].arrive()
            yield
            if add:
                while min(stored) < it + 1:
                    yield

    def mma():
        kv, st, pt, nq = 0, [0, 0], [0, 0], 0

        def scores(i, j, kv, ns, n):
            k = kv + 2 * j

            def do():
                assert stage[k % NS] == k, "scores of another tile"
            pipe.append(do)
            bar = s_full[i][st[i] & 1]
            pipe.append(bar.arrive)
            st[i] += 1
            if i == 1 or j >= ns[1]:
                pipe.append(empty[k % NS].arrive)
                if j + 1 == n:
                    pipe.append(q_empty.arrive)
        it = -1
        while True:
            it += 1
            yield from wait(item_full[it % ITEMS], it // ITEMS)
            assert slot[it % (2 * ITEMS)] == it
            item_empty[it % ITEMS].arrive()
            yield
            if it == len(items):
                return
            n0, n1, whole = ns = items[it]
            n = max(n0, n1)
            if n == 0:
                continue
            yield from wait(q_full, nq)
            nq += 1
            got = set()

            def need(t):
                yield from wait(full[t % NS], t // NS)
                got.add(t)

            def sc(i, j):
                if kv + 2 * j not in got:
                    yield from need(kv + 2 * j)
                scores(i, j, kv, ns, n)
            if n0:
                yield from sc(0, 0)
            if n1:
                yield from sc(1, 0)
            if bufs == 3 and n0 > 1:
                yield from sc(0, 1)
            for j in range(n):
                v = kv + 2 * j + 1
                yield from need(v)
                for i in range(2):
                    if j < ns[i]:
                        yield from wait(p_ready[i][pt[i] & 1], pt[i] >> 1)

                        def do(v=v, j=j, whole=whole):
                            assert stage[v % NS] == v, "P V of another tile"
                            assert j < whole or looked[v] == LOOKS, "P V before the look"
                        pipe.append(do)
                        pipe.append(o_done[i][pt[i] & 1].arrive)
                        pt[i] += 1
                    if i == 0:
                        if (bufs == 2 and j + 1 < n0) or (bufs == 3 and j + 1 < n1):
                            yield from sc(0 if bufs == 2 else 1, j + 1)
                pipe.append(empty[v % NS].arrive)
                if bufs == 2 and j + 1 < n1:
                    yield from sc(1, j + 1)
                if bufs == 3 and j + 2 < n0:
                    yield from sc(0, j + 2)
                yield
            kv += 2 * n

    def softmax(i):
        t, it = 0, -1
        while True:
            it += 1
            yield from wait(item_full[it % ITEMS], it // ITEMS)
            assert slot[it % (2 * ITEMS)] == it
            item_empty[it % ITEMS].arrive()
            yield
            if it == len(items):
                return
            for _ in range(items[it][i]):
                yield from wait(s_full[i][t & 1], t >> 1)
                yield
                p_ready[i][t & 1].arrive()
                t += 1
            if items[it][i]:
                yield from wait(o_done[i][(t - 1) & 1], (t - 1) >> 1)
            yield
            stored[i] = it + 1

    roles = [tma(), mma(), softmax(0), softmax(1)] + [look() for _ in range(LOOKS)]
    weight = [r.choice((1, 1, 1, 5, 30)) for _ in roles]
    steps = 0
    while roles:
        steps += 1
        assert steps < 400000, "the roles wait for one another"
        x = r.random()
        if later and x < 0.2:
            later.pop(r.randrange(len(later)))()
        elif pipe and x < 0.5:
            pipe.popleft()()
        else:
            i = r.choices(range(len(roles)), weight)[0]
            try:
                next(roles[i])
            except StopIteration:
                del roles[i], weight[i]
    assert not later and set(stored) == {len(items)}


def some_items(r):
    out = []
    for _ in range(r.choice((1, 3, 12, 30))):
        n1 = r.choice((0, 0, 1, 1, 2, 3, 5, 9))
        n0 = max(0, n1 - r.choice((0, 0, 1)))
        out.append((n0, n1, max(0, max(n0, n1) - r.choice((0, 1, 1, 2, 3)))) if r.random() < 0.8 else (n1, 0, max(0, n1 - 1)))
    return out


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("seed", range(40))
def test_any_order(D, seed):
    run(some_items(random.Random(seed)), D, seed)


def failures(**planted):
    n = 0
    for seed in range(20):
        try:
            run([(3, 3, 2), (2, 2, 1), (4, 4, 2)] * 3, 64, seed, **planted)
        except AssertionError:
            n += 1
    return n


def test_the_model_sees_planted_mistakes():
    """A look that takes a job before its tile has landed; a job ring that is shorter than the tiles under way."""
    assert failures() == 0
    assert failures(unannounced=True) > 0
    assert failures(JOBS=2) > 0
