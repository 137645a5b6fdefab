"""Host-side refusals of the bounded-cache calls, through the C ABI (no GPU: nothing here is
enqueued)."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest

from paged_kv_cache_348_b200 import build as pbuild
from paged_kv_cache_348_b200 import pagedkv as pk

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    pbuild.build()
    return pk.load()


def window(lib, B=4, ql=1, Hq=8, Hkv=2, D=128, bs=16, M=4, N=64, W=8, S=0, scale=0.1, dtype=0,
           ptr=P(4096), ws=1 << 30):
    return lib.pa_decode_window(ptr, ptr, ptr, ptr, ptr, ptr, B, ql, Hq, Hkv, D, bs, M, N, W, S,
                                scale, dtype, ptr, ws, None, None)


def window8(lib, Hq=8, ql=1, W=8, sc=P(4096)):
    p = P(4096)
    return lib.pa_decode_window_e4m3_bs(p, p, p, p, sc, sc, p, p, 4, ql, Hq, 2, 128, 16, 4, 64, W,
                                        0, 0.1, 0, p, 1 << 30, None, None)


def prefill(lib, T=100, B=4, Hq=8, Hkv=2, D=128, bs=16, M=4, N=64, W=8, S=0, scale=0.1, dtype=0,
            ptr=P(4096), ws=256):
    return lib.pa_prefill_window(ptr, ptr, ptr, ptr, ptr, ptr, ptr, T, B, Hq, Hkv, D, bs, M, N, W,
                                 S, scale, dtype, ptr, ws, None, None)


def compact(lib, L=1, B=4, Hkv=2, D=128, elem=2, bs=16, N=64, K=8, sw=4, dw=4, ptr=P(4096),
            cache=4096):
    arr = (P * max(L, 1))(*[cache] * max(L, 1))
    return lib.pa_compact_tokens(arr, arr, L, ptr, sw, ptr, dw, ptr, ptr, ptr, K, 0, 0, B, Hkv, D,
                                 elem, bs, N, None, None)


INVALID, UNSUPPORTED, OK = pk.PA_ERR_INVALID, pk.PA_ERR_UNSUPPORTED, pk.PA_OK
HUGE = dict(N=1 << 27, bs=16)


def test_window(lib):
    for kw, rc in ((dict(W=0), INVALID), (dict(W=-5), INVALID), (dict(S=-1), INVALID),
                   (dict(ql=0), INVALID), (dict(ql=17), UNSUPPORTED), (dict(D=96), UNSUPPORTED),
                   (dict(bs=4), UNSUPPORTED), (dict(Hq=9), INVALID), (dict(dtype=3), UNSUPPORTED),
                   (dict(scale=float("inf")), INVALID), (dict(ptr=P(0)), INVALID),
                   (dict(ptr=P(4104)), INVALID), (dict(B=0), OK), (dict(B=-1), INVALID),
                   (HUGE, INVALID), (dict(M=1 << 28), INVALID)):
        assert window(lib, **kw) == rc, kw
    assert window8(lib, W=0) == INVALID
    assert window8(lib, sc=P(0)) == INVALID
    assert window8(lib, Hq=16, ql=3) == UNSUPPORTED            # 24 rows over 8-bit pools


def test_prefill(lib):
    for kw, rc in ((dict(W=0), INVALID), (dict(S=-1), INVALID), (dict(T=-1), INVALID),
                   (dict(D=96), UNSUPPORTED), (dict(bs=4), UNSUPPORTED), (dict(Hq=9), INVALID),
                   (dict(Hq=258, Hkv=2), UNSUPPORTED), (dict(dtype=3), UNSUPPORTED),
                   (dict(scale=float("nan")), INVALID), (dict(ptr=P(0)), INVALID),
                   (dict(ptr=P(4104)), INVALID), (dict(ws=100), INVALID), (dict(B=0), OK),
                   (dict(T=0), OK), (HUGE, INVALID), (dict(T=1 << 29), INVALID),
                   (dict(M=1 << 27), INVALID)):
        assert prefill(lib, **kw) == rc, kw
    assert lib.pa_prefill_workspace_bytes() == 256


def test_compact(lib):
    for kw, rc in ((dict(L=-1), INVALID), (dict(L=0), OK), (dict(B=0), OK), (dict(K=0), OK),
                   (dict(K=-1), INVALID), (dict(D=96), UNSUPPORTED), (dict(elem=4), UNSUPPORTED),
                   (dict(bs=4), UNSUPPORTED), (dict(sw=0), INVALID), (dict(dw=0), INVALID),
                   (dict(ptr=P(0)), INVALID), (dict(cache=4104), INVALID),
                   (dict(cache=0), INVALID), (HUGE, INVALID), (dict(sw=1 << 28), INVALID)):
        assert compact(lib, **kw) == rc, kw


def test_wrappers_refuse_what_is_not_an_int():
    for bad in (1.0, "8", None):
        with pytest.raises(pk.PagedKVError):
            pk._whole(bad, "window")
    assert pk._whole(np.int64(5), "window") == 5
    assert pk._whole(1 << 60, "window") == 0x7fffffff and pk._whole(-(1 << 60), "w") == -1
