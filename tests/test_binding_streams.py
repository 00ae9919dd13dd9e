"""Which stream a call without one goes to, with and without torch's short way to its handle."""
import types

import pytest
import torch

from w4a16_dequant_gemm_group_amd import binding as B


def test_a_torch_without_the_short_way(monkeypatch):
    monkeypatch.setattr(B, "_raw_stream", None)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: types.SimpleNamespace(cuda_stream=77))
    assert B._stream(None) == 77
    assert B._stream(types.SimpleNamespace(cuda_stream=5)) == 5 and B._stream(9) == 9


@pytest.mark.gpu
def test_both_ways_name_the_same_stream(monkeypatch):
    side = torch.cuda.Stream()
    short = [B._stream(None)]
    with torch.cuda.stream(side):
        short.append(B._stream(None))
    assert short == [torch.cuda.current_stream().cuda_stream, side.cuda_stream]
    monkeypatch.setattr(B, "_raw_stream", None)
    with torch.cuda.stream(side):
        assert B._stream(None) == side.cuda_stream
    assert B._stream(None) == short[0]
