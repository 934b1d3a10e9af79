"""The stream that a call runs on: the one given, as an object or a handle, or torch's current one, also with a torch that
offers no short way to its handle."""
import types

import pytest
import torch

import count_sketch_aggregation_amd as s2r


def test_given_streams():
    assert s2r._stream(0) == 0 and s2r._stream(77) == 77
    assert s2r._stream(types.SimpleNamespace(cuda_stream=1234)) == 1234


def test_current_stream_by_the_public_call(monkeypatch):
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: types.SimpleNamespace(cuda_stream=4321))
    assert s2r._stream(None) == 4321


@pytest.mark.gpu
def test_both_ways_name_the_same_stream(monkeypatch):
    side = torch.cuda.Stream()
    for stream in (torch.cuda.current_stream(), side):
        with torch.cuda.stream(stream):
            short = s2r._stream(None)
            with monkeypatch.context() as m:
                m.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
                assert s2r._stream(None) == short == stream.cuda_stream
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        assert s2r._stream(None) == torch.cuda.current_stream().cuda_stream
        torch.zeros(4, device="cuda")
