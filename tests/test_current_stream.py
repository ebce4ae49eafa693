"""The stream a call takes when none is given: the current stream's handle, by torch's public
interface where the shorter private one is missing."""
import types

import pytest
import torch

import bit_diffusion_amd as bd


def test_without_the_private_function(monkeypatch):
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: types.SimpleNamespace(cuda_stream=1234))
    assert bd._stream(None) == 1234


def test_with_it(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 5000 + device, raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    assert bd._stream(None) == 5003


def test_given_streams():
    assert bd._stream(0) == 0 and bd._stream(77) == 77
    assert bd._stream(types.SimpleNamespace(cuda_stream=99)) == 99


@pytest.mark.gpu
def test_both_name_the_same_stream(monkeypatch):
    side = torch.cuda.Stream()
    for stream in (torch.cuda.current_stream(), side):
        with torch.cuda.stream(stream):
            private = bd._stream(None)
            with monkeypatch.context() as m:
                m.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
                assert bd._stream(None) == private == stream.cuda_stream
