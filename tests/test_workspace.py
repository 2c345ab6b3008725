"""Where a Workspace's memory comes from, without a GPU: streams are stand-ins
that record which of them is current when memory is allocated."""

import contextlib
import gc
import weakref

import pytest
import torch

pytest.importorskip("newton_schulz_dmuon_amd")
from newton_schulz_dmuon_amd import api  # noqa: E402


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle
        self.capturing = False


class Buffer:
    def __init__(self, owner, nbytes):
        self.owner, self.nbytes, self.users, self.device = owner, nbytes, [], torch.device("cuda", 0)

    def numel(self):
        return self.nbytes

    def record_stream(self, stream):
        self.users.append(stream)


@pytest.fixture
def streams(monkeypatch):
    current = [Stream(1)]

    @contextlib.contextmanager
    def use(s):
        current.append(s)
        yield
        current.pop()

    monkeypatch.setattr(torch.cuda, "stream", use)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: current[-1])
    monkeypatch.setattr(torch, "empty", lambda n, dtype, device: Buffer(current[-1], n))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: current[-1].capturing)
    monkeypatch.setattr(api, "_raw_stream", lambda index: current[-1].cuda_stream)
    return current


DEVICE = torch.device("cuda", 0)


def test_memory_belongs_to_the_stream_that_uses_it(streams):
    s = Stream(2)
    assert api.Workspace().get(1000, DEVICE).owner is streams[0]
    ws = api.Workspace()
    buf = ws.get(1000, DEVICE, s)
    assert buf.owner is s and not buf.users and len(streams) == 1
    assert ws.get(10, DEVICE, s) is buf and not buf.users
    assert ws.get(2000, DEVICE, s).owner is s


def test_a_device_without_an_index_is_the_current_one(streams):
    ws = api.Workspace()
    buf = ws.get(1000, "cuda")
    assert buf.numel() == 1000 and ws.get(1000, torch.device("cuda")) is buf
    assert ws.get(1000, DEVICE) is buf and ws.get(1000, "cuda:0") is buf


def test_other_streams_are_recorded(streams):
    s = Stream(2)
    ws = api.Workspace()
    buf = ws.get(1000, DEVICE, s)
    assert ws.get(1000, DEVICE) is buf and buf.users == [streams[0]]
    ws = api.Workspace()
    buf = ws.get(1000, DEVICE)
    assert ws.get(500, DEVICE, s) is buf and buf.users == [s]
    with torch.cuda.stream(s):
        assert ws.get(500, DEVICE) is buf and buf.users == [s, s]


@pytest.mark.parametrize("other", [False, True])
def test_a_captured_buffer_is_kept(streams, other):
    """Warmed, captured, then grown by an eager call: the graph still writes the
    first buffer."""
    s = Stream(2) if other else None
    ws = api.Workspace()
    first = weakref.ref(ws.get(1000, DEVICE, s))
    (s or streams[0]).capturing = True
    ws.get(1000, DEVICE, s)
    ws.get(800, DEVICE, s)
    (s or streams[0]).capturing = False
    second = weakref.ref(ws.get(2000, DEVICE, s))
    assert ws.get(4000, DEVICE, s).numel() == 4000
    gc.collect()
    assert first() is not None and second() is None  # the second was in no capture
    del ws
    gc.collect()
    assert first() is None
