"""CPU: which stream the binding's calls take when none is given, on a torch with and without its raw-handle function."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")


class Stream:
    cuda_stream = 0x5eed


@pytest.fixture
def q8(monkeypatch):
    import q8_block_quantized_02_b200 as m
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: Stream())
    return m


def test_raw_handle_of_the_current_device(q8, monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0x1000 + device, raising=False)
    assert q8._stream(None) == 0x1003


def test_without_the_raw_handle_function(q8, monkeypatch):
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    assert q8._stream(None) == 0x5eed


def test_given_streams(q8):
    assert q8._stream(7) == 7 and q8._stream(Stream()) == 0x5eed
