"""A CPU model of how lora_attn_chunk's roles end when a wait runs out (csrc/attn_chunk.cu): the watch declares the CTA failed
at any point, or a copy never lands and it does so for that. Every role then ends within a few more waits, nobody reads a
piece that was not published or that is being overwritten, no converting warp is left at the four's barrier, and the items
that the CTA has a part of are marked so that the join leaves them. Variants that break one rule each are caught."""
from __future__ import annotations

import os
import random
import re

import pytest

SRC = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gather_lora_gb300", "csrc",
                        "attn_chunk.cu")).read()
RING, STAGES, TAKERS, SOFT = 4, 2, 4, 2        # pieces in the ring, stages of key tiles, converting warps, softmax warps of the model


class Barrier:
    def __init__(self, count):
        self.count, self.pending, self.phase = count, count, 0

    def arrive(self):
        self.pending -= 1
        if self.pending == 0:
            self.phase, self.pending = self.phase + 1, self.count

    def passed(self, phase):                    # the phase-th completion (0: the first) has been; parity as the hardware tests it
        return (self.phase & 1) != (phase & 1)


class Broken(AssertionError):
    pass


def run(pieces, seed, fail_at=None, lost=None, rule=None):
    """pieces: key tiles of each. fail_at: the scheduler's step at which the watch fires; lost: the key tile whose copy never
    lands (the watch fires when nothing moves). rule: None, or the rule that this variant breaks."""
    r = random.Random(seed)
    failed = [False]
    full, empty = [Barrier(1) for _ in range(RING)], [Barrier(SOFT + 2 + TAKERS) for _ in range(RING)]
    landed, ready, free = [Barrier(1) for _ in range(STAGES)], [Barrier(TAKERS) for _ in range(STAGES)], [Barrier(1) for _ in range(STAGES)]
    scores, weights = [Barrier(1) for _ in range(2)], [Barrier(SOFT) for _ in range(2)]
    slot = [None] * RING                        # what a slot of the ring holds: (piece, tiles), None: never published
    vote = dict(n=0, any=False, round=0, out=[])
    busy = [0] * RING                           # roles that are reading the slot

    def wait(bar, phase):                       # -> True: failed
        while not bar.passed(phase):
            if failed[0]:
                return True
            yield
        return False

    def piece(it):                              # -> tiles, or None: the end, or failed
        yield from wait(full[it % RING], it // RING)
        if failed[0] and rule != "pieces are read after a failure":
            return None
        if slot[it % RING] is None or slot[it % RING][0] != it:
            raise Broken(f"piece {it} is read, its slot holds {slot[it % RING]}")
        return slot[it % RING][1]

    def planner():
        for it in range(len(pieces) + 1):
            if it >= RING:
                yield from wait(empty[it % RING], it // RING - 1)
            if failed[0]:
                if rule == "a piece is published after a failure":
                    if busy[it % RING]:
                        raise Broken("a slot is overwritten while it is read")
                    slot[it % RING] = (it, 0)
                    full[it % RING].arrive()
                return
            if busy[it % RING]:
                raise Broken("a slot is overwritten while it is read")
            slot[it % RING] = (it, pieces[it] if it < len(pieces) else 0)
            full[it % RING].arrive()
            yield

    def use(it):
        busy[it % RING] += 1

    def leave(it):
        busy[it % RING] -= 1
        empty[it % RING].arrive()

    def loader():
        kt, it = 0, 0
        while True:
            n = yield from piece(it)
            if not n:
                return
            use(it)
            for j in range(n):
                k = kt + j
                if k >= STAGES:
                    yield from wait(free[k % STAGES], k // STAGES - 1)
                if failed[0]:
                    break
                if k != lost:
                    landed[k % STAGES].arrive()
                yield
            kt += n
            leave(it)
            it += 1

    def together():                             # the four's barrier with its vote -> someone saw the failure
        vote["any"] |= failed[0]
        vote["n"] += 1
        mine = vote["round"]
        if vote["n"] == TAKERS:
            vote["out"].append(vote["any"])
            vote.update(n=0, any=False, round=mine + 1)
        while len(vote["out"]) <= mine:
            yield "barrier"
        return vote["out"][mine] if rule != "each converting warp decides for itself" else failed[0]

    def taker():
        kt, it = 0, 0
        while True:
            n = yield from piece(it)
            if rule != "no vote at a piece" and (yield from together()):
                return
            if not n:
                return
            use(it)
            for j in range(n):
                k = kt + j
                yield from wait(landed[k % STAGES], k // STAGES)
                if (yield from together()):
                    break
                ready[k % STAGES].arrive()
                yield
            kt += n
            leave(it)
            it += 1

    def mma():
        kt, it = 0, 0
        while True:
            n = yield from piece(it)
            if not n:
                return
            use(it)
            dead = False
            for j in range(n):
                k = kt + j
                dead |= yield from wait(ready[k % STAGES], k // STAGES)
                scores[k & 1].arrive()
                dead |= yield from wait(weights[k & 1], k >> 1)
                free[k % STAGES].arrive()
                if dead:
                    break
                yield
            kt += n
            leave(it)
            it += 1

    stored = []

    def softmax():
        kt, it = 0, 0
        while True:
            n = yield from piece(it)
            if not n:
                return
            use(it)
            for j in range(n):
                dead = yield from wait(scores[(kt + j) & 1], (kt + j) >> 1)
                if dead:
                    break
                weights[(kt + j) & 1].arrive()
                yield
            kt += n
            if not failed[0]:
                stored.append(it)
            leave(it)
            it += 1

    agents = [planner(), loader(), mma()] + [taker() for _ in range(TAKERS)] + [softmax() for _ in range(SOFT)]
    live, still, step, after = list(range(len(agents))), 0, 0, 0
    while live:
        step += 1
        if step == fail_at or (still > 400 and not failed[0]):
            failed[0], still = True, 0
        if failed[0]:
            after += 1
            # (a turn of the scheduler is at most one wait of a role; a piece is a few)
            if after > 200 * len(agents):
                raise Broken(f"roles {live} go on after the failure")
        a = r.choice(live)
        was = [b.phase for b in full + empty + landed + ready + free + scores + weights] + [vote["round"]]
        try:
            next(agents[a])
        except StopIteration:
            live.remove(a)
        now = [b.phase for b in full + empty + landed + ready + free + scores + weights] + [vote["round"]]
        still = 0 if was != now else still + 1
        if step > 100000:
            raise Broken("no end")
    return failed[0], stored


@pytest.mark.parametrize("seed", range(60))
def test_every_role_ends(seed):
    r = random.Random(seed)
    pieces = [r.randint(1, 9) for _ in range(r.randint(0, 14))]
    bad, stored = run(pieces, seed)
    assert not bad and sorted(stored) == sorted(list(range(len(pieces))) * SOFT)
    for k in range(40):
        run(pieces, seed * 100 + k, fail_at=r.randint(1, 60 * (len(pieces) + 1)))
    if pieces:
        for k in range(20):
            lost = r.randrange(sum(pieces))
            bad, stored = run(pieces, seed * 100 + k, lost=lost)
            assert bad
            at = next(i for i in range(len(pieces)) if lost < sum(pieces[:i + 1]))
            assert all(i < at for i in stored)


@pytest.mark.parametrize("rule", ["pieces are read after a failure", "each converting warp decides for itself", "no vote at a piece",
                                  "a piece is published after a failure"])
def test_broken_rules_are_caught(rule):
    caught = 0
    for seed in range(150):
        r = random.Random(seed)
        pieces = [r.randint(1, 9) for _ in range(r.randint(3, 14))]
        try:
            run(pieces, seed, fail_at=r.randint(1, 600), rule=rule)
        except Broken:
            caught += 1
    assert caught > 0, rule


def body(begin, end):
    at = SRC.index(begin)
    return SRC[at:SRC.index(end, at)]


def test_the_kernel_keeps_these_rules():
    """The places of the source that the model stands for."""
    # one wait for a piece, whose answer is asked before the piece is
    assert len(re.findall(r"wait\(c, c\.piece_full", SRC)) == 1
    here = body("bool piece_here(", "\n}")
    assert re.search(r"__any_sync\(0xffffffffu, failed\(c\)\) && c\.piece\[it % kPieces\]\.valid", here)
    assert len(re.findall(r"piece_here\(c, it\)", SRC)) == 5      # look-up, converting, token-by-token loading, MMA, softmax warps
    assert "valid) break" not in SRC.replace("if (!valid) break", "")
    # all slots of the ring begin without a piece
    assert "c.piece[i].valid = 0" in body("mbar_init(smem_u32(&c.ended)", "mbar_fence_init")
    # the planning warp leaves without publishing
    plan = body("for (int it = 0;; ++it) {\n      const int sl = it % kPieces;\n      // (a slot", "c.piece[sl] = w")
    assert re.search(r"if \(__any_sync\(0xffffffffu, failed\(c\)\)\) break;", plan) and "mbar_wait_limit" not in plan
    # the converting warps leave together: at a piece, and at a tile before the second barrier
    take = body("Warp q of the four has rows", "// =========================== K and V tiles")
    assert len(re.findall(r"takers_failed\(c\)", take)) == 2 and len(re.findall(r"takers_sync\(\)", take)) == 1
    assert take.index("gone = takers_failed(c)") < take.index("takers_sync()")
    # what a failed CTA left in the workspace is not joined
    assert "kGone" in body("atomicOr(&g_chunk_status", "if (warp == kMmaWarp)")
    join = SRC[SRC.index("chunk_join_kernel("):]
    assert join.index("if (s_gone) return") < join.index("p.lse[") and join.index("if (s_gone) return") < join.index("p.out +")
