"""lora_attn_chunk with the smallest and with large scales, over windows whose first tile some rows do not see (-m gpu)."""
from __future__ import annotations

import pytest

import test_gpu_attn_chunk as C
from gather_lora_gb300 import lib as L
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    require_gpu()
    L.lora_read_device_status(clear=True)
    yield
    assert L.lora_read_device_status(clear=True) == 0


@pytest.mark.parametrize("fmt", C.FMTS)
@pytest.mark.parametrize("scale", [2.0 ** -140, 2.0 ** -126, 2.0 ** -60, 30.0])
@pytest.mark.parametrize("d,kv,G,page", [(64, 1, 1, 16), (128, 2, 4, 20)])
def test_scales(fmt, scale, d, kv, G, page):
    data = C.case(d + G, [(300, 1500), (40, 9000), (5, 5), (200, 260)], kv, G, d, page, fmt, spread=0.2 if scale > 1 else 1.0)
    for window, sinks in ((200, 0), (130, 3), (1000, 0)):
        C.compare(*data, kv * G, scale, window, sinks)
