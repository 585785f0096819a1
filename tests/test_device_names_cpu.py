"""Devices given as names: the binding takes "cuda:1" as it takes 1 and torch.device("cuda", 1)."""
import contextlib

import pytest
import torch

from transformer_xl_relative_attn_gb300 import _lib


@pytest.fixture
def two_devices(monkeypatch):
    """Device 0 is current; what is asked of torch.cuda is recorded."""
    seen = []

    class Stream:
        cuda_stream = 99

    def raw(index):
        assert type(index) is int, f"ordinal is {index!r}"
        return 100 + index

    def entered(device):
        seen.append(device)
        return contextlib.nullcontext()

    monkeypatch.setattr(_lib, "_raw_stream", raw)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream())
    monkeypatch.setattr(torch.cuda, "device", entered)
    monkeypatch.setitem(_lib._functions, "probe", lambda *args: args)
    return seen


@pytest.mark.parametrize("device,handle", [(1, 101), ("cuda:1", 101), (torch.device("cuda", 1), 101), ("cuda:0", 100),
                                           ("cuda", 99), (torch.device("cuda"), 99)])
def test_current_stream_of_a_device(two_devices, device, handle):
    assert _lib._stream(None, device) == handle


@pytest.mark.parametrize("device", [0, "cuda:0", torch.device("cuda", 0)])
def test_current_device_is_not_entered_again(two_devices, device):
    assert _lib._invoke(device, "probe", 7) == (7,) and two_devices == []


@pytest.mark.parametrize("device", [1, "cuda:1", torch.device("cuda", 1), "cuda", torch.device("cuda")])
def test_other_devices_are_entered(two_devices, device):
    assert _lib._invoke(device, "probe", 7) == (7,) and two_devices == [device]
