"""The binding's Workspace and what its calls make for themselves, without a GPU."""
from __future__ import annotations

import weakref

import pytest
import torch

import w4a16_group_quantized_gb300 as w4


@pytest.mark.parametrize("name", ["get", "get_scratch"])
def test_an_outgrown_buffer_is_kept(name):
    """A call that is still running, or a captured graph, uses it."""
    ws = w4.Workspace("cpu")
    grow, first = getattr(ws, name), weakref.ref(ws.buf if name == "get" else ws.scratch)
    grow(1000)
    second = weakref.ref(grow(1000))
    assert grow(1 << 16).numel() >= 1 << 16
    assert first() is not None and second() is not None
    total = sum(b.numel() for b in ws._outgrown)
    assert total < grow(0).numel() and grow(1).data_ptr() == grow(1 << 16).data_ptr()


def test_what_a_call_makes_is_made_on_its_stream(monkeypatch):
    inside = []

    class On:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            inside.append(self.stream)

        def __exit__(self, *exc):
            inside.pop()

    made = []

    def spy(real):
        def f(*a, **kw):
            made.append(inside[-1] if inside else None)
            return real(*a, **kw)
        return f

    ws = w4.Workspace("cpu")
    monkeypatch.setattr(torch.cuda, "stream", On)
    monkeypatch.setattr(torch, "empty", spy(torch.empty))
    monkeypatch.setattr(torch, "zeros", spy(torch.zeros))
    ws.get(1000, "side")
    ws.get_scratch(1000, "side")
    assert made == ["side", "side"]
    made.clear()
    ws.get_scratch(1 << 20)
    assert made == [None]
    made.clear()
    recorded = []
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: "current")
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: recorded.append(s))
    t = w4._empty((2, 3), torch.float16, "cpu", "side")
    assert t.shape == (2, 3) and made == ["side"] and recorded == ["current"]
    w4._empty((2, 3), torch.float16, "cpu", None)
    assert made == ["side", None] and recorded == ["current"]
