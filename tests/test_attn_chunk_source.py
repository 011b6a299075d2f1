"""Orderings in csrc/attn_chunk.cu that no result shows reliably, read from its source."""
from __future__ import annotations

import os

SRC = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gather_lora_gb300", "csrc",
                        "attn_chunk.cu")).read()


def test_the_plans_sums_are_fenced_from_the_copies_that_overwrite_them():
    """The sums of the plan lie where TMA brings the first K tile. Ordinary accesses to shared memory come before those of the
    asynchronous proxy only if a proxy fence stands between them, in the threads that made them and before the barrier."""
    plan = SRC[SRC.index("long long* const sums = "):SRC.index("if (warp == kPlanWarp)")]
    assert "base + Sm::ring" in plan.split(";")[0]
    last_use, last_barrier = plan.rindex("sums["), plan.rindex("__syncthreads()")
    assert last_use < plan.rindex("fence_proxy_async_smem()") < last_barrier
