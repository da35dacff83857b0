"""The binding's first use, which several threads may make at once (no GPU)."""
import sys

import pytest

from variable_length_prefill_gb300 import _binding as B


def test_nothing_is_seen_half_made(monkeypatch):
    """A thread takes a set _torch_module for everything being there, so at
    every line of the first use's setup it is unset, or all the rest is set."""
    pytest.importorskip("torch")
    rest = ("_i32", "_types", "_raw_stream", "_device", "_take", "_give")
    for name in rest + ("_torch_module",):
        monkeypatch.setattr(B, name, None)
    half = []

    def look(frame, event, arg):
        if frame.f_code is not B._torch.__code__:
            return None
        if B._torch_module is not None:
            half.extend((frame.f_lineno, n) for n in rest if getattr(B, n) is None)
        return look

    before = sys.gettrace()
    sys.settrace(look)
    try:
        B._torch()
    finally:
        sys.settrace(before)
    assert B._torch_module is not None and not half, half
