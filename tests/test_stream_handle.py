"""The stream handle a call passes on: the current stream's, by torch's undocumented quick way or
without it, or the given one's (CPU: torch's calls replaced)."""
from __future__ import annotations

import types

import torch

from paged_kv_cache_348_b200 import pagedkv as pk


def test_current_stream_with_and_without_the_undocumented_name(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream",
                        lambda: types.SimpleNamespace(cuda_stream=0x5000))
    monkeypatch.setattr(pk, "_raw_stream", lambda device: 0x1000 + device)
    assert pk._stream(None) == 0x1003
    monkeypatch.setattr(pk, "_raw_stream", None)
    assert pk._stream(None) == 0x5000


def test_given_streams():
    assert pk._stream(types.SimpleNamespace(cuda_stream=0x77)) == 0x77
    assert pk._stream(0x88) == 0x88 and pk._stream(0) == 0
