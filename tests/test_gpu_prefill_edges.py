"""pa_prefill_window at the ends of its range: bad pages inside tiles without a mask, groups of up
to 128 query heads."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from paged_kv_cache_348_b200 import pagedkv as pk
from tests import window_ref as ref
from tests.helpers import bits, from_bits
from tests.test_gpu_prefill import MIX, expect, run, setup

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D,bs", [(64, 1), (64, 8), (64, 16), (64, 32), (128, 1), (128, 8),
                                  (128, 16), (128, 32)])
def test_a_bad_page_reads_as_zeros(dtype, D, bs):
    """As in the decode calls: rows of a page with an id out of range are zeros.  Whatever the
    other sequences hold, the bits are the same."""
    mix = [(150, 150), (100, 900), (3, 700), (300, 600)]
    case, starts, q = setup(mix, 8, 2, D, bs, dtype, 5000, 0, D + bs, drop=False)
    case["tables"][1, 200 // bs] = -1
    case["tables"][1, 600 // bs:632 // bs] = case["N"]
    case["tables"][2, 0] = 1 << 30
    outs = []
    rng = np.random.default_rng(3)
    mine = np.zeros(case["N"], bool)
    for s in (1, 2):
        t = case["tables"][s]
        mine[t[(t >= 0) & (t < case["N"])]] = True
    for other in (1, 100):
        c = dict(case)
        for p in ("k", "v"):
            x = from_bits(case[p], dtype).clone()
            x[torch.from_numpy(~mine)] *= other
            x[torch.from_numpy(~mine)] = x[torch.from_numpy(~mine)].flip(0)
            c[p] = bits(x)
        for _ in range(2):
            out, st = run(c, starts, q, 5000, 0)
            assert st == pk.DEV_BAD_BLOCK_ID
            outs.append(out[starts[1]:starts[3]].view(torch.int16))
    for o in outs[1:]:
        assert torch.equal(o, outs[0])
    want, bound = expect(c, starts, q, 5000, 0)
    ref.check(out[starts[1]:starts[3]], want[starts[1]:starts[3]], bound[starts[1]:starts[3]])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D,bs", [(128, 16), (64, 1)])
@pytest.mark.parametrize("Hq,Hkv", [(43, 1), (128, 2), (65, 1), (142, 2), (100, 1), (128, 1),
                                    (256, 2)])
def test_large_groups(dtype, D, bs, Hq, Hkv):
    """33 to 128 query heads a kv head: subtiles of one to three tokens, rows left idle."""
    mix = [m for m in MIX if m[0] < 100] + [(70, 400)]
    case, starts, q = setup(mix, Hq, Hkv, D, bs, dtype, 100, 4, Hq + D)
    out, st = run(case, starts, q, 100, 4)
    assert st == 0
    ref.check(out, *expect(case, starts, q, 100, 4), "group %d" % (Hq // Hkv))


def test_group_past_the_range_is_refused():
    case, starts, q = setup([(4, 20)], 129, 1, 64, 16, "f16", 60, 4, 2)
    with pytest.raises(pk.PagedKVError):
        run(case, starts, q, 60, 4)
