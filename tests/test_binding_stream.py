"""The stream that a call of the binding enqueues on (CPU: the handles alone)."""
import types

import pytest
import torch

import moe_decode_tail_gb300 as mt


class Stream:
    cuda_stream = 4711


def test_a_given_stream_is_passed_on():
    assert mt._stream(Stream()) == 4711 and mt._stream(12) == 12 and mt._stream(0) == 0


@pytest.mark.parametrize("lost", ["_cuda_getCurrentRawStream", "_cuda_getDevice"])
def test_the_current_stream_without_torchs_private_functions(monkeypatch, lost):
    # a torch without one of them: the public call
    private = types.SimpleNamespace(_cuda_getCurrentRawStream=lambda device: 1, _cuda_getDevice=lambda: 0)
    monkeypatch.setattr(torch, "_C", private)
    assert mt._stream(None) == 1
    delattr(private, lost)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *device: Stream())
    assert mt._stream(None) == 4711


@pytest.mark.gpu
def test_the_current_stream_is_torchs():
    assert mt._stream(None) == torch.cuda.current_stream().cuda_stream
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        assert mt._stream(None) == side.cuda_stream == torch.cuda.current_stream().cuda_stream
    assert mt._stream(side) == side.cuda_stream
