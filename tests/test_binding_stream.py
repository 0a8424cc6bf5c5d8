"""The stream a binding call runs on, without a GPU."""

import types

import torch

from full_attention_decode_gb300 import binding as B


def test_no_stream_means_torchs_current_one(monkeypatch):
    """Asked for through torch's public API, with each call."""
    handles = iter([0x1230, 0])
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: types.SimpleNamespace(cuda_stream=next(handles)))
    assert B._stream(None) == 0x1230
    assert B._stream(None) == 0


def test_a_stream_or_its_handle_is_taken_as_it_is(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: 1 / 0)
    assert B._stream(0) == 0
    assert B._stream(77) == 77
    assert B._stream(types.SimpleNamespace(cuda_stream=99)) == 99
