"""pa_compact_tokens and pa_compact_tokens_e4m3_bs refuse a pool, or a scale array, that is named
twice: two walks over one pool in place would overwrite each other's rows (no GPU: nothing is
enqueued)."""
from __future__ import annotations

import ctypes

import pytest

from paged_kv_cache_348_b200 import build as pbuild
from paged_kv_cache_348_b200 import pagedkv as pk

P = ctypes.c_void_p
A, B, C, D = 1 << 20, 2 << 20, 3 << 20, 4 << 20


@pytest.fixture(scope="module")
def lib():
    pbuild.build()
    return pk.load()


def call(lib, k, v, ks=None, vs=None):
    arr = lambda x: (P * len(x))(*x)
    p = P(4096)
    scales = [] if ks is None else [arr(ks), arr(vs)]
    rest = [len(k), p, 4, p, 4, p, p, p, 8, 0, 0, 2, 2, 128]
    if ks is None:
        return lib.pa_compact_tokens(arr(k), arr(v), *rest, 2, 16, 64, None, None)
    return lib.pa_compact_tokens_e4m3_bs(arr(k), arr(v), *scales, *rest, 16, 64, None, None)


@pytest.mark.parametrize("k,v", [([A], [A]), ([A, A], [B, C]), ([A, B], [C, C]), ([A, B], [B, C])])
def test_pools(lib, k, v):
    assert call(lib, k, v) == pk.PA_ERR_INVALID
    assert call(lib, k, v, [A, B][:len(k)], [C, D][:len(k)]) == pk.PA_ERR_INVALID


@pytest.mark.parametrize("ks,vs", [([A, A], [B, C]), ([A, B], [C, B])])
def test_scale_arrays(lib, ks, vs):
    assert call(lib, [A, B], [C, D], ks, vs) == pk.PA_ERR_INVALID
