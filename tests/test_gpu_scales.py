"""Softmax scales of zero and below in the decode calls without a window, on both kernels (up to
8 and 9 to 64 query rows), and where the two meet in a cascade, against the 64-bit definition."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from paged_kv_cache_348_b200 import inputs
from paged_kv_cache_348_b200 import pagedkv as pk
from paged_kv_cache_348_b200 import workload as wl
from tests import window_ref as ref
from tests.helpers import bits, from_bits, make_case
from tests.test_gpu_cascade import GROUPS, run_cascade, shared_case
from tests.test_gpu_window import CTX, expected, u_p16

pytestmark = pytest.mark.gpu

SCALES = [0.0, -0.2]


def reference(case, q, u_p):
    dt = case["dtype"]
    k, v = (from_bits(case[x], dt).double() for x in ("k", "v"))
    return expected(case, from_bits(q, dt).double(), k, v, 1 << 20, 0, u_p)


def device(case):
    dt = case["dtype"]
    return (from_bits(case["k"], dt).cuda(), from_bits(case["v"], dt).cuda(),
            torch.from_numpy(np.ascontiguousarray(case["tables"])).cuda(),
            torch.from_numpy(case["ctx"]).cuda())


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("bs", [1, 16])
@pytest.mark.parametrize("Hq,q_len", [(4, 2), (3, 3), (16, 2), (8, 8)])
@pytest.mark.parametrize("scale", SCALES)
def test_several_new_tokens(dtype, bs, Hq, q_len, scale):
    case = make_case(len(CTX), Hq, 1, 128, bs, CTX, dtype=dtype, seed=12)
    case["scale"] = scale
    q = bits(inputs.randn((case["B"], q_len, Hq, 128), dtype, 3, stream=11))
    out = torch.full(q.shape, float("nan"), dtype=inputs.torch_dtype(dtype), device="cuda")
    st = pk.new_status()
    pk.pa_decode_multi(out, from_bits(q, dtype).cuda(), *device(case), scale,
                       pk.new_workspace(case["B"], Hq, 1, 128), st)
    assert int(st.item()) == 0
    ref.check(out, *reference(case, q, u_p16(dtype, Hq * q_len)), "multi")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("Hq", [4, 12, 64])
@pytest.mark.parametrize("scale", SCALES)
def test_fused_append_and_noalloc(dtype, Hq, scale):
    case = make_case(len(CTX), Hq, 1, 128, 16, CTX, dtype=dtype, seed=13)
    case["scale"] = scale
    q = case["q"].reshape(case["B"], 1, Hq, 128)
    want, bound = reference(case, q, u_p16(dtype, Hq))
    k, v, tab, ctx = device(case)
    qd = from_bits(case["q"], dtype).cuda()
    out = torch.full_like(qd, float("nan"))
    st = pk.new_status()
    # the newest tokens' rows go out of the cache and come back through the append
    new = []
    for pool in (k, v):
        rows = torch.zeros((case["B"], 1, 128), dtype=pool.dtype, device="cuda")
        for i, c in enumerate(case["ctx"]):
            if c:
                at = (int(case["tables"][i, (c - 1) // 16]), 0, (int(c) - 1) % 16)
                rows[i, 0] = pool[at]
                pool[at] = float("nan")
        new.append(rows)
    pk.pa_decode_append(out, qd, k, v, *new, tab, ctx, scale,
                        pk.new_workspace(case["B"], Hq, 1, 128), st)
    assert int(st.item()) == 0
    ref.check(out.unsqueeze(1), want, bound, "append")
    out.fill_(float("nan"))
    pk.pa_decode_noalloc(out, qd, k, v, tab, ctx, scale, st)
    assert int(st.item()) == 0
    ref.check(out.unsqueeze(1), want, bound, "noalloc")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("Hq,Hkv,width", [(8, 2, 2), (8, 2, 16), (16, 1, 4), (32, 8, 8)])
@pytest.mark.parametrize("scale", SCALES)
def test_cascade(dtype, Hq, Hkv, width, scale):
    """Chunks of 8 query rows (one kernel for both passes) and of 32 and 64 (the prefix on the
    tcgen05 kernel, the rest on the other)."""
    case = shared_case(GROUPS, Hq, Hkv, 128, 16, dtype, seed=14)
    case["scale"] = scale
    plan = wl.plan_cascade(case["tables"], case["ctx"], 16, Hq // Hkv, width)
    out, st, plan = run_cascade(case, plan)
    assert st == 0 and len(plan[2]) > 0
    q = case["q"].reshape(case["B"], 1, Hq, 128)
    # the coarser of the two passes' P; their join adds two 32-bit roundings to each
    want, bound = reference(case, q, max(u_p16(dtype, Hq // Hkv), u_p16(dtype, 64)) + 2.0 ** -22)
    ref.check(out.unsqueeze(1), want, bound, "cascade")
