"""The binding's Workspace, what its calls make for themselves and what they refuse, without a GPU."""
from __future__ import annotations

import weakref

import pytest
import torch

import w4a16_group_quantized_gb300 as w4
from w4a16_group_quantized_gb300 import build as w4build


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


def test_tensors_and_streams_of_another_device_are_refused(monkeypatch):
    """The library launches on the current device: handles of another one's streams or memory would run there."""
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 7, raising=False)

    class Stream:
        def __init__(self, index):
            self.device, self.cuda_stream = torch.device("cuda", index), 8 + index

    assert w4._handle(None, 0) == 7 and w4._handle(Stream(0), 0) == 8
    for stream, device in ((None, 1), (Stream(1), 1), (Stream(1), 0)):
        with pytest.raises(ValueError):
            w4._handle(stream, device)


def test_a_workspace_stays_on_its_device(monkeypatch):
    made = []
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch, "zeros", lambda *a, device=None, **kw: made.append(device))
    assert w4.Workspace().device == w4.Workspace("cuda").device == torch.device("cuda", 3)
    assert w4.Workspace("cuda:1").device == torch.device("cuda", 1)
    assert {str(d) for d in made} == {"cuda:3", "cuda:1"}


def test_experts_options_are_checked():
    w4build.build()
    lib = w4.load()
    at = 0x10000  # an aligned address that no refused call reads
    args = w4._EXPERTS_ARGS.pack(at, at, at, at, at, at, 0, 64, 64, 4, 2, 64, 1)  # no rows: nothing is enqueued

    def status(**kw):
        return lib.w4a16_experts_opts(args, at, 1 << 40, w4.ctypes.byref(w4.Options(**kw)), None)

    assert lib.w4a16_experts_opts(args, at, 1 << 40, None, None) == 0
    assert status() == status(flags=w4.FLAG_TEST_TIMEOUT, wait_limit_cycles=5) == 0
    for kw in (dict(flags=w4.FLAG_WEIGHTS_STATIC), dict(flags=8), dict(kernel=1), dict(block_n=64), dict(ctas=1), dict(schedule=1),
               dict(cluster=2), dict(dtype=1), dict(reserved=1)):
        assert status(**kw) == 1, kw
