"""Kept rows that cannot be moved (a position or a page out of range) in pools with block
scales: they are left out, the others of their block keep their values, whatever place the
rows left out have in it."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from paged_kv_cache_348_b200 import pagedkv as pk
from tests import window_ref as ref
from tests.test_gpu_compact import dev, setup

pytestmark = pytest.mark.gpu


def value(code):
    return torch.from_numpy(code).view(torch.float8_e4m3fn).double()


def reference(pool, scales, c, bs, layer):
    """Codes and scales after the call: a new block's scale is the one its first moved row
    fixes, rows that cannot be moved leave their place as it was."""
    new, ns = pool.copy(), scales.copy()
    N, Hkv = scales.shape
    for s in range(len(c["ctx"])):
        for h in range(Hkv):
            k = c["keep"][min(layer, c["keep"].shape[0] - 1), s, min(h, c["keep"].shape[2] - 1)]
            set_by = {}
            for i in range(c["n"][s]):
                t, j = int(k[i]), i // bs
                if not 0 <= t < c["ctx"][s]:
                    continue
                sb, db = int(c["src"][s, t // bs]), int(c["dst"][s, j])
                if not (0 <= sb < N and 0 <= db < N):
                    continue
                x = value(pool[sb, h, t % bs]) * float(scales[sb, h])
                if j not in set_by:
                    set_by[j] = ns[db, h] = ref.block_scale(float(x.abs().max()))
                y = ref.quantise_e4m3(x / float(ns[db, h]))
                new[db, h, i % bs] = y.float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    return new, ns


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bs", [1, 8, 16, 32])
@pytest.mark.parametrize("what", ["position", "source page", "page"])
def test_rows_left_out(in_place, D, bs, what):
    L, Hkv, ctx = 2, 2, [200, 333, 77, 150]
    c = setup(L, Hkv, D, bs, D + bs, in_place, True, True, 0.6, ctx)
    status = pk.DEV_BAD_KEEP
    if what == "position":
        # at a block's start, inside one, a run over a whole block, the last row
        for s, rows in ((0, [0]), (1, [3, 32]), (2, list(range(0, 33))), (3, [89, 64, 65, 66])):
            for i in rows:
                c["keep"][:, s, :, i] = (-1, ctx[s], 1 << 30)[i % 3]
    else:
        status = pk.DEV_BAD_BLOCK_ID
        t = c["src"] if what == "source page" else c["dst"]
        t[0, 0], t[1, 1], t[2, -1 if t is c["dst"] else 2] = -1, c["N"], 1 << 30
    pools, scales = [], []
    for _ in range(2 * L):
        x = torch.from_numpy(c["rng"].normal(0, 20, (c["N"], Hkv, bs, D))).clamp(-448, 448)
        pools.append(x.float().to(torch.float8_e4m3fn).view(torch.uint8).numpy())
        scales.append(np.exp2(c["rng"].integers(-12, 6, (c["N"], Hkv))).astype(np.float32))
    tens = [torch.from_numpy(p).cuda() for p in pools]
    sct = [torch.from_numpy(s).cuda() for s in scales]
    st = pk.new_status()
    pk.pa_compact_tokens_e4m3_bs(tens[:L], tens[L:], sct[:L], sct[L:], *dev(c), st)
    assert int(st.item()) == status
    for i, t in enumerate(tens):
        want, ns = reference(pools[i], scales[i], c, bs, i % L)
        assert torch.equal(sct[i].cpu(), torch.from_numpy(ns)), "scales of pool %d" % i
        got = t.cpu().numpy()
        # codes as numbers (0 and -0 are the same value)
        assert torch.equal(value(got), value(want)), np.argwhere(got != want)[0]
