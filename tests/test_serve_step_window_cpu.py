"""The example layer's window on the CPU: what its calls could not take is refused when the layer is made."""
from __future__ import annotations

import pytest

from gather_lora_gb300 import lib as L
from test_serve_step_cpu import layer


def test_windows_that_no_call_takes_are_refused():
    for kw in (dict(window=0), dict(window=-3), dict(window=2 ** 31), dict(window=2 ** 40), dict(sinks=-1), dict(sinks=2 ** 31), dict(window=4, sinks=2 ** 33)):
        with pytest.raises(ValueError, match="window"):
            layer(**kw)
    assert layer(window=None).window == layer(window=L.NO_WINDOW).window == L.NO_WINDOW
    assert layer(window=L.NO_WINDOW - 1, sinks=L.NO_WINDOW).sinks == L.NO_WINDOW
