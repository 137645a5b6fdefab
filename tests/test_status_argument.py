"""The status argument of the bounded-cache calls: int32 on the current device with an element, or
none (CPU: stand-ins for device tensors; nothing is enqueued)."""
from __future__ import annotations

import pytest
import torch

from paged_kv_cache_348_b200 import pagedkv as pk


class OnDevice:
    """What the checks ask of a tensor."""

    def __init__(self, dtype=torch.int32, n=1, device=0, cuda=True):
        self.dtype, self.n, self.index, self.is_cuda = dtype, n, device, cuda
        self.device = "cuda:%d" % device

    def is_contiguous(self):
        return True

    def dim(self):
        return 1

    def numel(self):
        return self.n

    def get_device(self):
        return self.index if self.is_cuda else -1


def test_status(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    t = OnDevice(torch.float16, 8)
    pk._here("call", None, t)
    pk._here("call", OnDevice(), t)
    pk._here("call", OnDevice(n=4), t)
    for bad in (OnDevice(torch.uint8, 4), OnDevice(torch.int64), OnDevice(torch.float32),
                OnDevice(n=0), OnDevice(device=1), OnDevice(cuda=False)):
        with pytest.raises(pk.PagedKVError):
            pk._here("call", bad, t)
    with pytest.raises(pk.PagedKVError):
        pk._here("call", None, t, OnDevice(device=1))
