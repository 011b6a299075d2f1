"""lora_rope_init's table against exact arithmetic: every entry is the nearest to its angle, so that far positions keep
their angles (-m gpu for the rotation itself)."""
from __future__ import annotations

import ctypes
import os
import random
from fractions import Fraction

import pytest
import torch

import attn_util as A
import step_refs as S
import test_gpu_rope as T
from gather_lora_gb300 import lib as L
from gpu_util import require_gpu

# pi to 100 digits
PI = Fraction(31415926535897932384626433832795028841971693993751058209749445923078164062862089986280348253421170680, 10 ** 100)
FREQS = [1.0, 0.5, 10000.0 ** -0.75, 1e-9, 6.283185307179586, 1234.5, -0.3, -1e-22, 3e5, 0.1, 2.0 ** -40, 2.0 ** 40, -7.7e9, 1e15, 1.7e19, 2.0 ** 64 - 2.0 ** 11,
         3.0, -6.283185307179586, 2.0 ** -64, 1e-300, 5e-324, 0.0, 500000.0 ** -0.5, 1.0 - 2.0 ** -53]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not os.path.exists(L.LIB_PATH):
        from gather_lora_gb300 import build
        build.build()
    L.load()


def part(x):
    """A number's fraction, as its distance from the nearest whole one."""
    x = x % 1
    return min(x, 1 - x)


def test_every_entry_is_the_nearest():
    r = random.Random(1)
    for freqs in (FREQS, [r.choice((-1, 1)) * 2.0 ** r.uniform(-70, 63.9) for _ in range(24)], [10000.0 ** (-j / 24) for j in range(24)]):
        turns = L.Rope(128, rotary_dim=48, freqs=freqs).struct.turns
        for f, t in zip(freqs, turns):
            # half a unit, and less than 2^-64 units for what the constant leaves out
            assert part(Fraction(int(t), 2 ** 64) - Fraction(f) / (2 * PI)) <= Fraction(1, 2 ** 65) + Fraction(1, 2 ** 128), f


def test_frequencies_that_the_table_cannot_hold_are_refused():
    for f in (2.0 ** 64, -2.0 ** 64, 1e300, float("inf"), float("-inf"), float("nan")):
        r = L._RopeStruct()
        r.axes = 77
        assert L.load().lora_rope_init(ctypes.byref(r), 128, 8, (ctypes.c_double * 4)(1.0, f, 1.0, 1.0), None, 1, 0) == -2 and r.axes == 77
        assert "freqs[1]" in L.lora_last_error()


@pytest.mark.gpu
@pytest.mark.parametrize("inter", [False, True])
def test_far_positions_keep_their_angles(inter):
    """Frequencies of every size to the ends of int32, the whole turns taken off in exact arithmetic."""
    require_gpu()
    d, n = 64, 200
    freqs = (FREQS + [base ** (-j / 8) for base in (10000.0, 500000.0) for j in range(4)])[:32]
    g, r = A.gen(2), random.Random(3)
    pos = [2 ** 31 - 1, -2 ** 31, -1, 0, 1, 2 ** 24 + 1] + [r.choice((-1, 1)) * int(2 ** r.uniform(0, 31)) for _ in range(n - 6)]
    angle = torch.tensor([[float(Fraction(p) * Fraction(f) / (2 * PI) % 1) for f in freqs] for p in pos], dtype=torch.float64, device="cuda")[:, None] * 2 * torch.pi
    rows = A.randn(g, n, 3 * d)
    out = torch.empty_like(rows)
    L.lora_qk_rope(rows, 3 * d, out, 3 * d, None, 0, None, 0, n, 3, 0, L.Rope(d, freqs=freqs, interleaved=inter), A.int32(pos), n)
    x = rows.double().view(n, 3, d)
    x0, x1 = (x[..., 0::2], x[..., 1::2]) if inter else (x[..., :32], x[..., 32:])
    y0, y1, mag = x0 * angle.cos() - x1 * angle.sin(), x1 * angle.cos() + x0 * angle.sin(), x0.abs() + x1.abs()
    join = (lambda a, b: torch.stack((a, b), -1).flatten(-2)) if inter else (lambda a, b: torch.cat((a, b), -1))
    # (S.F32 holds the fp32 steps; the angle's own 2^-31 turns are 2^-28)
    T.within(out, join(y0, y1), join(mag, mag) * (1 + 2.0 ** -28 / S.F32), inter)
