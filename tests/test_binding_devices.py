"""Where the calls that pass through the C module run: on their tensors' device,
whichever is current.  The devices are stand-ins, so no GPU is needed."""
from __future__ import annotations

from contextlib import contextmanager
from types import SimpleNamespace

import pytest
import torch

from paged_kv_cache_355_b200 import build


@pytest.fixture
def devices(monkeypatch):
    """Device 0 is current; records the device that is current at each call."""
    build.build()
    from paged_kv_cache_355_b200 import _binding as b

    seen = SimpleNamespace(current=[0], calls=[], status=0, entered=0)

    @contextmanager
    def device(index):
        seen.entered += 1
        seen.current.append(index)
        try:
            yield
        finally:
            seen.current.pop()

    def call(entry, index, dtype, args):
        seen.calls.append((entry, index, seen.current[-1]))
        return seen.status

    monkeypatch.setattr(torch.cuda, "current_device", lambda: seen.current[-1])
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 1000 + index, raising=False)
    monkeypatch.setattr(b, "_marshal", SimpleNamespace(call=call))
    return b, seen


def test_the_call_runs_on_its_tensors_device(devices):
    b, seen = devices
    for index in (0, 3):
        b._call(b._SELECT, index, None, ())
    assert seen.calls == [(b._SELECT, 0, 0), (b._SELECT, 3, 3)]
    assert seen.entered == 1 and seen.current == [0]  # no switch for the current device, and back afterwards


def test_back_on_the_current_device_after_an_error(devices):
    b, seen = devices
    seen.status = 1
    with pytest.raises(b.PAError, match="pa_block_scores failed: PA_ERR_INVALID_ARG"):
        b._call(b._SCORES, 2, None, ())
    seen.status = -1
    with pytest.raises(TypeError, match="scores must be a CUDA tensor"):
        b._call(b._SELECT, 2, None, (torch.zeros(1),))
    assert seen.current == [0]


def test_the_stream_is_that_devices(devices, monkeypatch):
    b, _ = devices
    assert b._raw_stream(None, 0) == 1000 and b._raw_stream(None, 3) == 1003
    assert b._raw_stream(None, -1) == 0           # a CPU tensor, refused by name later

    class Stream:
        device = SimpleNamespace(index=1)
        cuda_stream = 77

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    assert b._raw_stream(Stream(), 1) == 77
    with pytest.raises(ValueError, match="the stream belongs to"):
        b._raw_stream(Stream(), 0)
