"""The stream a binding call runs on."""

import types

import pytest
import torch

from full_attention_decode_gb300 import binding as B

from harness import init


def test_no_stream_means_torchs_current_one(monkeypatch):
    """Asked for with each call, of torch's public API where the shorter way is not there."""
    monkeypatch.setattr(B, "_raw_stream", None)
    handles = iter([0x1230, 0])
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: types.SimpleNamespace(cuda_stream=next(handles)))
    assert B._stream(None) == 0x1230
    assert B._stream(None) == 0


def test_no_stream_means_the_current_devices_current_one(monkeypatch):
    device = iter([0, 1, 0])
    monkeypatch.setattr(torch.cuda, "current_device", lambda: next(device))
    monkeypatch.setattr(B, "_raw_stream", lambda d: 0x100 + d)
    assert [B._stream(None) for _ in range(3)] == [0x100, 0x101, 0x100]


def test_a_stream_or_its_handle_is_taken_as_it_is(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: 1 / 0)
    monkeypatch.setattr(B, "_raw_stream", lambda d: 1 / 0)
    assert B._stream(0) == 0
    assert B._stream(77) == 77
    assert B._stream(types.SimpleNamespace(cuda_stream=99)) == 99


@pytest.mark.gpu
def test_both_ways_name_the_same_stream(monkeypatch):
    init()
    for st in (torch.cuda.default_stream(), torch.cuda.Stream()):
        with torch.cuda.stream(st):
            short = B._stream(None)
            with monkeypatch.context() as m:
                m.setattr(B, "_raw_stream", None)
                assert B._stream(None) == short == st.cuda_stream
