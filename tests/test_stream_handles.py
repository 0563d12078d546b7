"""The handle of the current stream, with torch's function for it and without."""
import types

import pytest
import torch

import gated_delta_rule_45_amd as kda
from gated_delta_rule_45_amd import gdn

NAME = "_cuda_getCurrentRawStream"


def test_torch_without_the_function(monkeypatch):
    monkeypatch.delattr(torch._C, NAME, raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda index: types.SimpleNamespace(cuda_stream=0x70 + index))
    assert gdn._current_handle(3) == 0x73


def test_torch_with_the_function(monkeypatch):
    monkeypatch.setattr(torch._C, NAME, lambda index: 0x50 + index, raising=False)
    assert gdn._current_handle(2) == 0x52


@pytest.mark.gpu
@pytest.mark.parametrize("there", [True, False])
def test_calls_go_to_the_current_stream(monkeypatch, there):
    if not there:
        monkeypatch.delattr(torch._C, NAME, raising=False)
    s = torch.cuda.Stream()
    for stream in (torch.cuda.current_stream(), s):
        with torch.cuda.stream(stream):
            assert gdn._current_handle(0) == stream.cuda_stream
    q, freq = torch.randn(1, 5, 2, 64, device="cuda:0"), kda.rope_frequencies(64, device="cuda:0")[0]
    want, _ = kda.rope(q, None, freq)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):  # (a launch on another stream than the capture's would run now and not in the replay)
        y, _ = kda.rope(q, None, freq)
    y.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want)
