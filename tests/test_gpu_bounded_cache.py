"""The bounded-cache operators together, as a serving loop uses them: prompts appended and
attended, pages behind the window given back and reused, tokens decoded, a fork, and the kept
tokens compacted; every step against the 64-bit definition over the tokens that each sequence
should see."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from paged_kv_cache_348_b200 import inputs
from paged_kv_cache_348_b200 import pagedkv as pk
from paged_kv_cache_348_b200.block_manager import BlockManager
from tests import window_ref as ref

pytestmark = pytest.mark.gpu

WINDOW, SINKS = 70, 5


class Server:
    """One layer of a model with a bounded cache; `rows` are the true K/V of every sequence."""

    def __init__(self, dtype, bs, Hq=8, Hkv=2, D=64, blocks=90):
        self.dt, self.bs, self.Hq, self.Hkv, self.D = dtype, bs, Hq, Hkv, D
        self.t = inputs.torch_dtype(dtype)
        self.g = torch.Generator().manual_seed(bs)
        self.bm = BlockManager(blocks, bs, inputs.pool_order(blocks, 3))
        nan = torch.full((blocks, Hkv, bs, D), float("nan"), dtype=self.t, device="cuda")
        self.k, self.v = nan, nan.clone()
        self.rows = {}
        self.ws, self.pws = pk.new_workspace(4, Hq, Hkv, D), pk.new_prefill_workspace()
        self.st = pk.new_status()
        self.scale = D ** -0.5

    def rand(self, *shape):
        return torch.randn(shape, generator=self.g).to(self.t)

    def append(self, sids, counts):
        """New tokens of each sequence into the cache, copy-on-write included."""
        slots, pairs, ks, vs = [], [], [], []
        for s, n in zip(sids, counts):
            k, v = self.rand(n, self.Hkv, self.D), self.rand(n, self.Hkv, self.D)
            old = self.rows.get(s)
            self.rows[s] = (k, v) if old is None else (torch.cat([old[0], k]), torch.cat([old[1], v]))
            for _ in range(n):
                slot, cow = self.bm.append_token(s)
                slots.append(slot)
                if cow:
                    pairs.append(cow)
            ks.append(k)
            vs.append(v)
        if pairs:
            pk.pa_copy_blocks([self.k], [self.v], torch.tensor(pairs, dtype=torch.int32).cuda(),
                              self.st)
        if slots:
            pk.pa_cache_append(self.k, self.v, torch.cat(ks).cuda(), torch.cat(vs).cuda(),
                               torch.tensor(slots, dtype=torch.int64).cuda(), self.st)

    def tables(self, sids):
        return (torch.from_numpy(self.bm.block_tables(sids, fill=-9)).cuda(),
                torch.from_numpy(self.bm.context_lens(sids)).cuda())

    def expect(self, s, q, u_p):
        k, v = (x.double() for x in self.rows[s])
        pos = torch.arange(len(k) - len(q), len(k))
        return ref.attend(q.double(), k, v, pos, WINDOW, SINKS, self.scale, u_p, self.dt)

    def prefill(self, sids, counts):
        self.append(sids, counts)
        q = self.rand(sum(counts), self.Hq, self.D)
        starts = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        out = torch.empty_like(q, device="cuda")
        pk.pa_prefill_window(out, q.cuda(), self.k, self.v, *self.tables(sids),
                             torch.from_numpy(starts).cuda(), WINDOW, SINKS, self.scale, self.pws,
                             self.st)
        for i, s in enumerate(sids):
            a, b = starts[i], starts[i + 1]
            ref.check(out[a:b], *self.expect(s, q[a:b], ref.U_OUT[self.dt]), "prefill %d" % s)
        self.trim(sids)

    def decode(self, sids, new=1):
        self.append(sids, [new] * len(sids))
        q = self.rand(len(sids), new, self.Hq, self.D)
        out = torch.empty_like(q, device="cuda")
        pk.pa_decode_window(out, q.cuda(), self.k, self.v, *self.tables(sids), WINDOW, SINKS,
                            self.scale, self.ws, self.st)
        u_p = 2.0 ** -16 if self.dt == "bf16" else 2.0 ** -11
        for i, s in enumerate(sids):
            ref.check(out[i], *self.expect(s, q[i], u_p), "decode %d" % s)
        self.trim(sids)

    def trim(self, sids):
        """Pages behind the window go back to the pool; what they held is overwritten."""
        before = {s: self.bm.table(s) for s in sids}
        for s in sids:
            self.bm.drop_window(s, WINDOW, SINKS)
        for s in sids:
            for b, c in zip(before[s], self.bm.table(s)):
                if b >= 0 and c < 0 and self.bm.refcount(b) == 0:
                    self.k[b] = float("nan")
                    self.v[b] = float("nan")

    def compact(self, sids, keeps):
        tables, ctx = self.tables(sids)
        dst = torch.from_numpy(self.bm.compact(sids, [len(k) for k in keeps])).cuda()
        keep = torch.zeros((1, len(sids), 1, max(map(len, keeps))), dtype=torch.int32)
        for i, x in enumerate(keeps):
            keep[0, i, 0, :len(x)] = torch.tensor(x)
        n = torch.tensor([len(k) for k in keeps], dtype=torch.int32).cuda()
        pk.pa_compact_tokens([self.k], [self.v], tables, dst, ctx, keep.cuda(), n, self.st)
        for s, x in zip(sids, keeps):
            self.rows[s] = tuple(r[torch.tensor(x)] for r in self.rows[s])


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("bs", [1, 8, 16, 32])
def test_serving_loop(dtype, bs):
    sv = Server(dtype, bs, blocks=1440 // bs)
    a, b = sv.bm.allocate(0), sv.bm.allocate(0)
    sv.prefill([a, b], [300, 33])
    sv.prefill([a, b], [101, 150])                  # the next chunk of both
    for _ in range(3):
        sv.decode([a, b])
    c = sv.bm.fork(a)                               # shares a's pages, gone ones included
    sv.rows[c] = sv.rows[a]
    sv.decode([a, b, c], new=4)
    assert sv.bm._L.pa_bm_num_blocks_of(sv.bm._h, a) < len(sv.bm.table(a)) or bs == 32
    # the visible tokens of each, a few of the window left out
    lens = {s: len(sv.rows[s][0]) for s in (a, b, c)}
    keeps = [list(range(SINKS)) + [t for t in range(lens[s] - WINDOW, lens[s]) if t % 5]
             for s in (a, c)]
    sv.compact([a, c], keeps)
    sv.decode([a, b, c])
    sv.prefill([c, a], [90, 1])
    for _ in range(2):
        sv.decode([a, b, c])
    assert int(sv.st.item()) == 0
    held = {x for s in (a, b, c) for x in sv.bm.table(s) if x >= 0}
    assert sv.bm.free_blocks + len(held) == 1440 // bs


def test_compacting_forks_together_over_8_bit_pages():
    """Two sequences that share pages, compacted in one call: both get fresh pages, the third
    keeps the shared ones; decode over the block-scaled pools sees the kept tokens."""
    Hq, Hkv, D, bs, n = 8, 2, 128, 16, 100
    bm = BlockManager(60, bs)
    g = torch.Generator().manual_seed(7)
    a = bm.allocate(n)
    b, c = bm.fork(a), bm.fork(a)
    k8, v8 = (torch.full((60, Hkv, bs, D), 0x7f, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.full((60, Hkv), float("nan"), device="cuda") for _ in range(2))
    kn, vn = (torch.randn((n, Hkv, D), generator=g).half().cuda() for _ in range(2))
    slots = torch.tensor([bm.slot_of(a, t) for t in range(n)], device="cuda")
    pk.pa_cache_append_e4m3_bs(k8, v8, ks, vs, kn, vn, slots)

    def values(s, count):
        out = []
        for p, sc in ((k8, ks), (v8, vs)):
            p, sc = p.view(torch.float8_e4m3fn).double().cpu(), sc.double().cpu()
            t = [bm.slot_of(s, i) for i in range(count)]
            out.append(torch.stack([p[x // bs, :, x % bs] * sc[x // bs][:, None] for x in t]))
        return out

    before = values(a, n)
    keeps = [list(range(0, n, 3)), [1, 2, 50, 99]]
    tables = torch.from_numpy(bm.block_tables([a, b])).cuda()
    ctx = torch.from_numpy(bm.context_lens([a, b])).cuda()
    dst = bm.compact([a, b], [len(x) for x in keeps])
    assert not set(dst[dst > 0]) & set(bm.table(c))
    keep = torch.zeros((1, 2, 1, len(keeps[0])), dtype=torch.int32)
    for i, x in enumerate(keeps):
        keep[0, i, 0, :len(x)] = torch.tensor(x)
    st = pk.new_status()
    pk.pa_compact_tokens_e4m3_bs([k8], [v8], [ks], [vs], tables, torch.from_numpy(dst).cuda(), ctx,
                                 keep.cuda(), torch.tensor([len(x) for x in keeps],
                                                           dtype=torch.int32).cuda(), st)
    after_c = values(c, n)
    assert torch.equal(after_c[0], before[0]) and torch.equal(after_c[1], before[1])
    for s, x in ((a, keeps[0]), (b, keeps[1])):
        for got, old in zip(values(s, len(x)), before):
            # quantised once more: at most half a step of 2^-4 relative, or of the block's
            # smallest step (2^-9 scales, a scale at most a quarter of its block's values)
            assert bool(((got - old[x]).abs() <= old[x].abs() * 2.0 ** -4 + 2.0 ** -10).all())
    assert int(st.item()) == 0
    # decode sees the codes that are there
    q = torch.randn((2, Hq, D), generator=g).half()
    out = torch.empty((2, Hq, D), dtype=torch.float16, device="cuda")
    pk.pa_decode_window_e4m3_bs(out, q.cuda(), k8, v8, ks, vs,
                                torch.from_numpy(bm.block_tables([a, b])).cuda(),
                                torch.from_numpy(bm.context_lens([a, b])).cuda(), 20, 2, D ** -0.5,
                                pk.new_workspace(2, Hq, Hkv, D), st)
    for i, (s, x) in enumerate(((a, keeps[0]), (b, keeps[1]))):
        k, v = values(s, len(x))
        want, bound = ref.attend(q[i:i + 1].double(), k, v, torch.tensor([len(x) - 1]), 20, 2,
                                 D ** -0.5, 2.0 ** -11, "f16")
        ref.check(out[i:i + 1], want, bound)


def test_two_calls_at_once():
    """Prompt attention, windowed decode and a compaction on two streams at a time, a workspace
    each: the results that they give alone."""
    from tests.helpers import bits, from_bits, make_case

    ctx = [3000, 900, 64, 1, 2222, 17]
    case = make_case(6, 32, 8, 128, 16, ctx, dtype="bf16", seed=3, poison=False)
    k, v = (from_bits(case[x], "bf16").cuda() for x in ("k", "v"))
    tab, cl = torch.from_numpy(case["tables"]).cuda(), torch.from_numpy(case["ctx"]).cuda()
    n = [1500, 900, 1, 1, 700, 5]
    starts = torch.from_numpy(np.concatenate([[0], np.cumsum(n)]).astype(np.int32)).cuda()
    q = from_bits(bits(inputs.randn((sum(n), 32, 128), "bf16", 1, stream=1)), "bf16").cuda()
    qd = from_bits(bits(inputs.randn((6, 32, 128), "bf16", 1, stream=2)), "bf16").cuda()

    def prefill(ws, stream=None):
        out = torch.empty_like(q)
        pk.pa_prefill_window(out, q, k, v, tab, cl, starts, 500, 4, 0.09, ws, None, stream)
        return out

    def decode(ws, stream=None):
        out = torch.empty_like(qd)
        pk.pa_decode_window(out, qd, k, v, tab, cl, 500, 4, 0.09, ws, None, stream)
        return out

    want = prefill(pk.new_prefill_workspace()), decode(pk.new_workspace(6, 32, 8, 128))
    st = [torch.cuda.Stream() for _ in range(3)]
    pws = [pk.new_prefill_workspace() for _ in range(2)]
    dws = pk.new_workspace(6, 32, 8, 128)
    torch.cuda.synchronize()
    for _ in range(10):
        got = prefill(pws[0], st[0]), prefill(pws[1], st[1]), decode(dws, st[2])
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[0])
        assert torch.equal(got[2], want[1])


def test_offsets_past_32_bits():
    """Pages at the end of a 6.4 GB pool (K and V one tensor) and the same pages in a small one:
    the same bits from every operator."""
    bs, Hkv, D, big = 16, 8, 128, 200_000
    g = torch.Generator(device="cuda").manual_seed(1)
    ctx = torch.tensor([1000, 333], dtype=torch.int32, device="cuda")
    nb = [63, 21]
    pool = torch.empty((big, Hkv, bs, D), dtype=torch.bfloat16, device="cuda")
    small = torch.randn((90, Hkv, bs, D), generator=g, device="cuda").bfloat16()
    pool[-90:] = small
    tab = torch.zeros((2, 63), dtype=torch.int32, device="cuda")
    tab[0] = torch.randperm(90, generator=g, device="cuda")[:63].int()
    rest = torch.tensor(sorted(set(range(90)) - set(tab[0].tolist())), device="cuda").int()
    tab[1, :21] = rest[:21]
    starts = torch.tensor([0, 500, 520], dtype=torch.int32, device="cuda")
    q = torch.randn((520, 16, D), generator=g, device="cuda").bfloat16()
    qd = torch.randn((2, 16, D), generator=g, device="cuda").bfloat16()
    keep = torch.arange(3, 203, dtype=torch.int32, device="cuda").view(1, 1, 1, 200).expand(
        1, 2, 1, 200).contiguous()
    n = torch.tensor([200, 150], dtype=torch.int32, device="cuda")
    res = []
    for p, off in ((small, 0), (pool, big - 90)):
        t = (tab + off).contiguous()
        a, b = torch.empty_like(q), torch.empty_like(qd)
        pk.pa_prefill_window(a, q, p, p, t, ctx, starts, 300, 4, 0.09, pk.new_prefill_workspace())
        pk.pa_decode_window(b, qd, p, p, t, ctx, 300, 4, 0.09, pk.new_workspace(2, 16, Hkv, D))
        k2 = p if off else p.clone()
        pk.pa_compact_tokens([k2], [torch.zeros_like(k2)], t, t[:, :13].contiguous(), ctx, keep, n)
        res.append((a, b, k2[off:off + 90].clone() if off else k2))
    for x, y in zip(*res):
        assert torch.equal(x, y)
