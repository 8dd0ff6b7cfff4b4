"""Which device and stream a call of the binding runs on, with torch's own switches replaced by notes."""
import contextlib
from types import SimpleNamespace

import pytest
import torch

from kv_cache_compression_group_b200 import jolt as J


@pytest.fixture
def notes(monkeypatch):
    """What was made current, and for which calls, on a machine whose current device is 0."""
    log = []

    @contextlib.contextmanager
    def switch(to):
        log.append(to)
        yield
        log.append("back")
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    monkeypatch.setattr(torch.cuda, "device", switch)
    monkeypatch.setattr(torch.cuda, "stream", switch)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: ("current", device))
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device: (handle, device))

    @J._on_its_stream
    def call(x, y=2, stream=None):
        log.append((x.device, y, stream))
    return log, call


def on(device):
    return SimpleNamespace(device=torch.device(device))


@pytest.mark.parametrize("device", ["cuda", "cuda:0", "cpu"])
def test_the_current_device_is_left_alone(notes, device):
    log, call = notes
    call(on(device), 3)
    call(x=on(device), y=4)
    call(on(device), 5, None)
    assert log == [(torch.device(device), y, None) for y in (3, 4, 5)]


def test_another_device_is_made_current(notes):
    log, call = notes
    call(on("cuda:1"))
    assert log == [torch.device("cuda:1"), (torch.device("cuda:1"), 2, None), "back"]


@pytest.mark.parametrize("given,handle", [(4096, 4096), (SimpleNamespace(cuda_stream=64), 64), (0, 0), (1, 0), (2, 2)])
@pytest.mark.parametrize("device,want", [("cuda", "cuda:0"), ("cuda:1", "cuda:1")])
def test_a_given_stream_is_made_current(notes, given, handle, device, want):
    log, call = notes
    for form in ("keyword", "place"):
        log.clear()
        if form == "keyword":
            call(x=on(device), stream=given)
        else:
            call(on(device), 2, given)
        assert log == [(handle, torch.device(want)), (torch.device(device), 2, None), "back"]
