"""The binding asks torch for the current stream's handle by a short cut that is
not part of torch's public interface, and does without it where it is missing."""
import importlib.util
import sys

import pytest
import torch

from grouped_gemm_02_amd import binding


def _reloaded(monkeypatch):
    spec = importlib.util.spec_from_file_location("binding_without_short_cut", binding.__file__)
    m = importlib.util.module_from_spec(spec)
    monkeypatch.setitem(sys.modules, spec.name, m)
    spec.loader.exec_module(m)
    return m


def test_binding_without_the_short_cut(monkeypatch):
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)

    class Stream:
        cuda_stream = 1234

    monkeypatch.setattr(torch.cuda, "is_available", lambda: True)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream())
    m = _reloaded(monkeypatch)
    assert m._stream(None) == 1234 and m._current_handle(0) == 1234
    assert m._stream(Stream()) == 1234 and m._stream(7) == 7


@pytest.mark.gpu
def test_handles_agree(monkeypatch):
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        short = binding._stream(None)
        monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
        assert short == _reloaded(monkeypatch)._stream(None) == side.cuda_stream
