"""The bound of tests/weight_refs.py on the CPU: weights of 11 significant bits keep it, weights of 8 do not."""
from __future__ import annotations

import numpy as np
import pytest

import weight_refs as W


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [4, 16])
def test_the_bound_tells_tf32_weights_from_bf16(fmt, d, G):
    q, rows = W.case(G + d, fmt, 2, G, d, [2, 3, 5, 9, 40])
    want, bound = W.want(q, rows, 0.1)
    assert (np.abs(W.with_weights_of(11, q, rows, 0.1) - want) <= bound).all()
    off = np.abs(W.with_weights_of(8, q, rows, 0.1) - want) > bound
    for b in range(len(rows) - 1):          # (in every sequence of a few tokens)
        assert off[b].any()
