"""A stream of another device than the tensors' is refused before anything is launched on it (its kernels would
run there, on addresses of this device). Stand-ins for two devices' streams: no GPU is needed."""
from types import SimpleNamespace

import pytest
import torch

from linear_cross_entropy_chunked_gb300 import _binding


def test_stream_of_another_device(monkeypatch):
    def entered(*args):
        raise AssertionError("the stream was entered")
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "device", entered)
    monkeypatch.setattr(torch.cuda, "stream", entered)
    for dev, other in ((0, 1), (1, 0)):
        stream = SimpleNamespace(device=torch.device("cuda", other), cuda_stream=1234)
        with pytest.raises(ValueError, match="stream belongs to"):
            with _binding._on(torch.device("cuda", dev), stream):
                pass


def test_stream_of_the_same_device(monkeypatch):
    stream = SimpleNamespace(device=torch.device("cuda", 0), cuda_stream=1234)
    log = []

    class Entered:
        def __init__(self, s):
            self.s = s

        def __enter__(self):
            log.append(self.s)

        def __exit__(self, *exc):
            log.append(None)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "stream", Entered)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: log[-1])
    with _binding._on(torch.device("cuda", 0), stream) as s:
        assert s == 1234
    assert log == [stream, None]
