"""Which torch stream a stream argument stands for (no GPU needed: torch's stream types are replaced)."""
import contextlib

import pytest
import torch

import block_scaled_fp8_grouped_amd as bs


class Stream:
    def __init__(self, cuda_stream):
        self.cuda_stream = cuda_stream


class External(Stream):
    def __init__(self, cuda_stream):
        # torch takes a zero handle for "none given" and makes a stream of its own
        super().__init__(cuda_stream or 0xBAD)


@pytest.fixture
def entered(monkeypatch):
    """The handles of the streams that are made current."""
    got = []

    @contextlib.contextmanager
    def stream(s):
        got.append(s.cuda_stream)
        yield

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", External)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda: Stream(0))
    monkeypatch.setattr(torch.cuda, "stream", stream)
    return got


class Handle:  # not torch's, as another library's stream object
    def __init__(self, cuda_stream):
        self.cuda_stream = cuda_stream


@pytest.mark.parametrize("given,handle", [(0, 0), (0x70, 0x70), (Stream(0x70), 0x70), (Stream(0), 0), (Handle(0), 0),
                                          (Handle(0x70), 0x70)])
def test_stream_made_current(entered, given, handle):
    with bs._on(given):
        pass
    assert entered == [handle]
    assert bs._stream(given) == handle
