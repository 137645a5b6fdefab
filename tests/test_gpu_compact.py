"""pa_compact_tokens and pa_compact_tokens_e4m3_bs: whole pools compared, bit for bit, with
the definition applied row by row on a copy."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from paged_kv_cache_348_b200 import pagedkv as pk
from tests import window_ref as ref

pytestmark = pytest.mark.gpu

CTX = [0, 1, 7, 16, 33, 200, 513, 900]


def setup(L, Hkv, D, bs, seed, in_place, per_layer, per_head, frac=0.5, ctx=CTX):
    rng = np.random.default_rng(seed)
    B = len(ctx)
    n = [max(1, int(c * frac)) if c else 0 for c in ctx]
    width = max(1, max(-(-c // bs) for c in ctx))
    dst_w = max(1, max(-(-x // bs) for x in n))
    blocks = sum(-(-c // bs) for c in ctx)
    fresh = 0 if in_place else sum(-(-x // bs) for x in n)
    N = blocks + fresh + 2
    order = rng.permutation(N)
    src = np.full((B, width), -5, np.int32)
    dst = np.full((B, dst_w), -9, np.int32)
    at = 0
    for i, c in enumerate(ctx):
        nb = -(-c // bs)
        src[i, :nb] = order[at:at + nb]
        at += nb
    for i, x in enumerate(n):
        nb = -(-x // bs)
        if in_place:
            dst[i, :nb] = src[i, :nb]
        else:
            dst[i, :nb] = order[at:at + nb]
            at += nb
    kmax = max(n)
    keep = np.full((L if per_layer else 1, B, Hkv if per_head else 1, kmax), -1, np.int32)
    for idx in np.ndindex(keep.shape[:3]):
        c = ctx[idx[1]]
        keep[idx][:n[idx[1]]] = np.sort(rng.permutation(c)[:n[idx[1]]])
    return dict(src=src, dst=dst, keep=keep, n=np.array(n, np.int32), ctx=np.array(ctx, np.int32),
                N=N, rng=rng)


def reference(pool, c, bs, layer, scales=None):
    """pool [N, Hkv, bs, D] (bytes or bit patterns; with scales: codes) after the call."""
    new, ns = pool.copy(), None if scales is None else scales.copy()
    Hkv = pool.shape[1]
    for s in range(len(c["ctx"])):
        for h in range(Hkv):
            k = c["keep"][min(layer, c["keep"].shape[0] - 1), s, min(h, c["keep"].shape[2] - 1)]
            for i in range(c["n"][s]):
                t = k[i]
                sb, db = c["src"][s, t // bs], c["dst"][s, i // bs]
                if scales is None:
                    new[db, h, i % bs] = pool[sb, h, t % bs]
                    continue
                x = torch.from_numpy(pool[sb, h, t % bs]).view(torch.float8_e4m3fn).double()
                x = x * float(scales[sb, h])
                if i % bs == 0:
                    ns[db, h] = ref.block_scale(float(x.abs().max()))
                y = ref.quantise_e4m3(x / float(ns[db, h]))
                new[db, h, i % bs] = y.float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    return new, ns


def dev(c):
    return [torch.from_numpy(c[x]).cuda() for x in ("src", "dst", "ctx", "keep", "n")]


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("D,elem", [(64, 1), (64, 2), (128, 1), (128, 2)])
@pytest.mark.parametrize("bs", [1, 8, 16, 32])
@pytest.mark.parametrize("per_layer,per_head,frac", [(False, False, 0.9), (True, True, 0.3),
                                                     (False, True, 1.0)])
def test_rows(in_place, D, elem, bs, per_layer, per_head, frac):
    L, Hkv = 2, 3
    c = setup(L, Hkv, D, bs, D + bs + elem, in_place, per_layer, per_head, frac)
    np_t = np.uint8 if elem == 1 else np.int16
    pools = [c["rng"].integers(0, 100, (c["N"], Hkv, bs, D)).astype(np_t) for _ in range(2 * L)]
    tens = [torch.from_numpy(p).cuda() for p in pools]
    if elem == 2:
        tens = [t.view(torch.bfloat16) for t in tens]
    st = pk.new_status()
    pk.pa_compact_tokens(tens[:L], tens[L:], *dev(c), st)
    assert int(st.item()) == 0
    for i, t in enumerate(tens):
        want, _ = reference(pools[i], c, bs, i % L)
        got = (t.view(torch.int16) if elem == 2 else t).cpu().numpy()
        assert np.array_equal(got, want), (i, np.argwhere(got != want)[0])


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("D,bs", [(64, 1), (64, 16), (128, 1), (128, 8), (128, 16), (128, 32)])
@pytest.mark.parametrize("per_head,frac", [(False, 0.9), (True, 0.4)])
def test_e4m3_block_scales(in_place, D, bs, per_head, frac):
    L, Hkv, ctx = 2, 2, [0, 1, 7, 33, 300]
    c = setup(L, Hkv, D, bs, D + bs, in_place, True, per_head, frac, ctx)
    pools, scales = [], []
    for _ in range(2 * L):
        sc = np.exp2(c["rng"].integers(-12, 6, (c["N"], Hkv))).astype(np.float32)
        x = torch.from_numpy(c["rng"].normal(0, 20, (c["N"], Hkv, bs, D))).clamp(-448, 448)
        x[c["rng"].integers(0, c["N"]), 0, 0] = 0        # a row of zeros sets scale 1
        pools.append(x.float().to(torch.float8_e4m3fn).view(torch.uint8).numpy())
        scales.append(sc)
    tens = [torch.from_numpy(p).cuda() for p in pools]
    sct = [torch.from_numpy(s).cuda() for s in scales]
    st = pk.new_status()
    pk.pa_compact_tokens_e4m3_bs(tens[:L], tens[L:], sct[:L], sct[L:], *dev(c), st)
    assert int(st.item()) == 0
    for i, t in enumerate(tens):
        want, ns = reference(pools[i], c, bs, i % L, scales[i])
        assert np.array_equal(sct[i].cpu().numpy(), ns)
        got = t.view(torch.float8_e4m3fn).float().cpu().numpy()
        assert np.array_equal(got, torch.from_numpy(want).view(torch.float8_e4m3fn).float().numpy())


def test_long_in_place_move_by_one():
    """Every row moves one position: each chunk's destination overlaps its source."""
    ctx = [20000, 4097]
    c = setup(1, 1, 128, 16, 3, True, False, False, 1.0, ctx)
    for s, x in enumerate(ctx):
        c["keep"][0, s, 0, :x - 1] = np.arange(1, x)
        c["n"][s] = x - 1
    pool = c["rng"].integers(0, 30000, (c["N"], 1, 16, 128)).astype(np.int16)
    k = torch.from_numpy(pool).cuda().view(torch.float16)
    v = k.clone()
    for _ in range(3):                                   # the same again, on the moved rows
        want, _ = reference(k.view(torch.int16).cpu().numpy(), c, 16, 0)
        pk.pa_compact_tokens([k], [v], *dev(c))
        assert np.array_equal(k.view(torch.int16).cpu().numpy(), want)
        assert torch.equal(k.view(torch.int16), v.view(torch.int16))


def test_bad_positions_counts_and_pages_are_reported_and_skipped():
    c = setup(1, 2, 64, 16, 8, False, False, False, 0.5, [100, 100, 100])
    pool = c["rng"].integers(0, 100, (c["N"], 2, 16, 64)).astype(np.int16)

    def run(c):
        k = torch.from_numpy(pool).cuda().view(torch.bfloat16)
        st = pk.new_status()
        pk.pa_compact_tokens([k], [k.clone()], *dev(c), st)
        return k.view(torch.int16).cpu().numpy(), int(st.item())

    good, st = run(c)
    assert st == 0
    b = dict(c, keep=c["keep"].copy())
    b["keep"][0, 1, 0, 3], b["keep"][0, 1, 0, 4] = -1, 100
    got, st = run(b)
    assert st == pk.DEV_BAD_KEEP
    blk = c["dst"][1, 0]
    assert np.array_equal(got[blk, :, 3:5], pool[blk, :, 3:5])       # left as they were
    got[blk, :, 3:5] = good[blk, :, 3:5]
    assert np.array_equal(got, good)
    assert run(dict(c, n=np.array([50, 999, -3], np.int32)))[1] == pk.DEV_BAD_KEEP
    src = c["src"].copy()
    src[0, 0] = c["N"]
    assert run(dict(c, src=src))[1] == pk.DEV_BAD_BLOCK_ID
    dst = c["dst"].copy()
    dst[2, 1] = -1
    assert run(dict(c, dst=dst))[1] == pk.DEV_BAD_BLOCK_ID
    assert run(dict(c, ctx=np.array([100, -1, 100], np.int32)))[1] == (
        pk.DEV_BAD_CONTEXT_LEN | pk.DEV_BAD_KEEP)


def test_refusals():
    c = setup(1, 2, 64, 16, 8, False, False, False, 0.5, [100, 100])
    k = torch.zeros((c["N"], 2, 16, 64), dtype=torch.bfloat16, device="cuda")
    src, dst, ctx, keep, n = dev(c)
    ok = [[k], [k.clone()], src, dst, ctx, keep, n]
    for at, bad in ((2, src[:1]), (3, dst.long()), (5, keep[0]), (6, n[:1]),
                    (5, keep.expand(1, 2, 3, -1).contiguous()), (0, [k, k]), (4, ctx.cpu())):
        args = list(ok)
        args[at] = bad
        with pytest.raises(pk.PagedKVError):
            pk.pa_compact_tokens(*args)
    with pytest.raises(pk.PagedKVError):
        pk.pa_compact_tokens([k[..., :32].contiguous()], [k[..., :32].contiguous()], *ok[2:])
    with pytest.raises(pk.PagedKVError):
        pk.pa_compact_tokens_e4m3_bs([k], [k], [k], [k], *ok[2:])
