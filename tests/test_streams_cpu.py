"""Which stream and device the Python layer gives its work to, on stand-ins for torch's streams (no GPU): a raw handle
is a stream of the device that the work is on, whichever device is current."""
import contextlib

import pytest
import torch

import diffusion_transformer_w4a4_b200 as svdq
from diffusion_transformer_w4a4_b200 import attention

SECOND = torch.device("cuda", 1)


class FakeStream:
    def __init__(self, handle, device=None):
        self.cuda_stream, self.device, self.stream_id = handle, device, handle


@pytest.fixture
def entered(monkeypatch):
    """The streams made current, in order; device 0 is the current device throughout."""
    seen = []

    @contextlib.contextmanager
    def current(stream):
        seen.append(stream)
        yield

    monkeypatch.setattr(torch.cuda, "Stream", FakeStream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", FakeStream)
    monkeypatch.setattr(torch.cuda, "stream", current)
    monkeypatch.setattr(torch.cuda, "device", lambda device: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: seen[-1])
    monkeypatch.setattr(attention, "_current_handle", lambda device: seen[-1].cuda_stream)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    return seen


def test_raw_handle_is_a_stream_of_the_works_device(entered):
    with svdq._stream_context(0x1234, SECOND):
        pass
    assert [(s.cuda_stream, s.device) for s in entered] == [(0x1234, SECOND)]


def test_handle_0_is_the_default_stream(entered, monkeypatch):
    default = FakeStream(0, SECOND)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device: default if device == SECOND else None)
    with svdq._stream_context(0, SECOND):
        pass
    assert entered == [default]


def test_attention_classes_take_the_raw_handle_to_their_device(entered):
    class Layer:
        N, K, device = 3 * 2 * 8, 16, SECOND

    to_out = Layer()
    to_out.N, to_out.K = 16, 16
    mod = attention.SelfAttention(Layer(), to_out, 2)
    with pytest.raises(ValueError, match="expected"):  # after the stream was made current
        mod(torch.zeros(3, 16), stream=0x55)
    assert [(s.cuda_stream, s.device) for s in entered] == [(0x55, SECOND)]


def test_stream_of_another_device_is_refused(entered):
    with pytest.raises(ValueError, match="stream of"):
        svdq._stream_context(FakeStream(7, torch.device("cuda", 0)), SECOND)
    assert not entered
