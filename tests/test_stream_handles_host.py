"""The stream argument as a handle (no GPU needed): results are allocated, and gradients run, on that very stream."""
import contextlib

import pytest
import torch

import dequant_iqk_moe_amd as q


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


@pytest.fixture
def entered(monkeypatch):
    """Handles of the streams that were made the current one; an external stream of handle 0 is a new one."""
    seen = []

    @contextlib.contextmanager
    def current(s):
        seen.append(s.cuda_stream)
        yield

    monkeypatch.setattr(torch.cuda, "stream", current)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: Stream(0))
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle: Stream(handle or 0xBAD))
    return seen


@pytest.mark.parametrize("given,handle", [(0, 0), (Stream(0), 0), (0x70, 0x70), (Stream(0x70), 0x70)])
def test_the_stream_of_a_handle(given, handle, entered):
    with q._on(given):
        pass
    assert q._empty((2, 3), torch.float32, "cpu", given).shape == (2, 3)
    assert q._stream(given).value == (handle or None)
    assert entered == [handle, handle]


def test_no_stream(entered):
    with q._on(None):
        pass
    q._empty((2,), torch.float32, "cpu", None)
    assert entered == []
