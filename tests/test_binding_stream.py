"""The stream that a call without one launches on."""
import types

import pytest
import torch

from deformable_convolution_sparse_b200 import binding as B


def test_without_the_undocumented_name_the_documented_ones_do(monkeypatch):
    monkeypatch.setattr(B, "_CURRENT_RAW_STREAM", None)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: types.SimpleNamespace(cuda_stream=4711))
    assert B._stream_handle(None) == 4711
    assert B._stream_handle(types.SimpleNamespace(cuda_stream=5)) == 5


@pytest.mark.gpu
def test_both_ways_name_the_current_stream(cuda_device, monkeypatch):
    s = torch.cuda.Stream()
    for raw in (B._CURRENT_RAW_STREAM, None):
        monkeypatch.setattr(B, "_CURRENT_RAW_STREAM", raw)
        assert B._stream_handle(None) == torch.cuda.current_stream().cuda_stream
        with torch.cuda.stream(s):
            assert B._stream_handle(None) == s.cuda_stream
