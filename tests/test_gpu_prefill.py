"""pa_prefill_window against the 64-bit definition: ragged chunks, masks, odd sizes, pages
given back, what lies outside every window poisoned with NaN, refusals."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from paged_kv_cache_348_b200 import inputs
from paged_kv_cache_348_b200 import pagedkv as pk
from tests import window_ref as ref
from tests.helpers import NAN_BITS, bits, from_bits, make_case
from tests.test_gpu_window import gathered, poison

pytestmark = pytest.mark.gpu

# (new tokens, context) of a batch: none, one, a whole prompt, a tail, more new tokens than
# positions, tiles of 128 rows and one more
MIX = [(0, 70), (1, 1), (37, 37), (5, 500), (3, 2), (64, 64), (129, 300), (0, 0), (1, 700),
       (200, 1029)]


def setup(mix, Hq, Hkv, D, bs, dtype, window, sinks, seed, drop=True, extra=3):
    case = make_case(len(mix), Hq, Hkv, D, bs, [c for _, c in mix], dtype=dtype, seed=seed,
                     poison=False)
    starts = np.zeros(len(mix) + 1, np.int32)
    starts[1:] = np.cumsum([n for n, _ in mix])
    # `poison` works for one number of new tokens: a sequence at a time
    hidden = np.ones((case["N"], bs), bool)
    for i, (n, _) in enumerate(mix):
        one = dict(case, B=1, tables=case["tables"][i:i + 1], ctx=case["ctx"][i:i + 1])
        hidden &= poison(one, n, window, sinks, drop)
    for p in ("k", "v"):
        case[p].transpose(0, 2, 1, 3)[hidden] = NAN_BITS[dtype]
    q = bits(inputs.randn((int(starts[-1]) + extra, Hq, D), dtype, seed, stream=11))
    return case, starts, q


def run(case, starts, q, window, sinks, scale=None, stream=None):
    dt = case["dtype"]
    out = torch.full(q.shape, 7.0, dtype=inputs.torch_dtype(dt), device="cuda")
    ws = pk.new_prefill_workspace()
    ws.fill_(0xFF)
    st = pk.new_status()
    pk.pa_prefill_window(out, from_bits(q, dt).cuda(), from_bits(case["k"], dt).cuda(),
                         from_bits(case["v"], dt).cuda(),
                         torch.from_numpy(np.ascontiguousarray(case["tables"])).cuda(),
                         torch.from_numpy(case["ctx"]).cuda(), torch.from_numpy(starts).cuda(),
                         window, sinks, case["scale"] if scale is None else scale, ws, st, stream)
    torch.cuda.synchronize()
    return out, int(st.item())


def expect(case, starts, q, window, sinks, scale=None):
    dt = case["dtype"]
    qd = from_bits(q, dt).double()
    k, v = (from_bits(case[x], dt).double() for x in ("k", "v"))
    want, bound = torch.full_like(qd, 7.0), torch.zeros_like(qd)
    for i in range(case["B"]):
        a, b = int(starts[i]), int(starts[i + 1])
        pos = torch.arange(int(case["ctx"][i]) - (b - a), int(case["ctx"][i]))
        # the weights are held in the cache's type when they meet V
        want[a:b], bound[a:b] = ref.attend(qd[a:b], gathered(case, i, k), gathered(case, i, v),
                                           pos, window, sinks,
                                           case["scale"] if scale is None else scale,
                                           ref.U_OUT[dt], dt)
    return want, bound


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D,bs", [(128, 16), (128, 32), (128, 8), (128, 1), (64, 16), (64, 32),
                                  (64, 8), (64, 1)])
@pytest.mark.parametrize("Hq,Hkv", [(4, 2), (3, 3), (10, 2), (16, 1)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (40, 4), (100, 33), (128, 0), (5000, 0),
                                          (300, 1)])
def test_shapes(dtype, D, bs, Hq, Hkv, window, sinks):
    case, starts, q = setup(MIX, Hq, Hkv, D, bs, dtype, window, sinks, D + bs + Hq + window)
    out, st = run(case, starts, q, window, sinks)
    assert st == 0
    ref.check(out, *expect(case, starts, q, window, sinks), "prefill_window")


def test_one_sequence_of_each_length():
    for n, ctx in ((1, 1), (2, 5), (31, 31), (32, 100), (33, 400), (255, 255), (256, 1000),
                   (257, 257), (1500, 2100)):
        case, starts, q = setup([(n, ctx)], 8, 1, 128, 16, "bf16", 200, 4, n, extra=0)
        out, st = run(case, starts, q, 200, 4)
        assert st == 0
        ref.check(out, *expect(case, starts, q, 200, 4), "n %d ctx %d" % (n, ctx))


def test_many_sequences_and_heads():
    """More items than CTAs, more sequences than a warp, lengths of zero among them."""
    rng = np.random.default_rng(0)
    mix = [(int(n), int(n) + int(p)) for n, p in zip(rng.integers(0, 90, 75),
                                                     rng.integers(0, 200, 75))]
    case, starts, q = setup(mix, 24, 8, 64, 16, "f16", 77, 3, 1)
    out, st = run(case, starts, q, 77, 3)
    assert st == 0
    ref.check(out, *expect(case, starts, q, 77, 3))
    for _ in range(3):                                    # whoever computes an item: same bits
        again, _ = run(case, starts, q, 77, 3)
        assert torch.equal(again, out)


@pytest.mark.parametrize("scale", [-0.2, 0.0, 3.0])
def test_scales(scale):
    case, starts, q = setup(MIX, 4, 2, 128, 16, "f16", 100, 4, 5)
    out, st = run(case, starts, q, 100, 4, scale=scale)
    assert st == 0
    ref.check(out, *expect(case, starts, q, 100, 4, scale=scale), "scale %g" % scale)


def test_scores_that_grow_move_the_reference():
    """Keys whose scores climb along the context: the maximum moves tile after tile."""
    case, starts, q = setup([(150, 1500)], 4, 2, 128, 16, "f16", 5000, 0, 5, extra=0)
    k = from_bits(case["k"], "f16")
    for b in range(-(-1500 // 16)):
        k[int(case["tables"][0, b])] *= b / 20
    case["k"] = bits(k)
    out, st = run(case, starts, q, 5000, 0)
    assert st == 0
    ref.check(out, *expect(case, starts, q, 5000, 0))


def test_agrees_with_decode():
    """The same new tokens through pa_decode_window: both within their bounds of one another."""
    case, starts, q = setup([(4, 900), (4, 77), (4, 4)], 8, 2, 128, 16, "f16", 150, 4, 2, extra=0)
    out, _ = run(case, starts, q, 150, 4)
    want, bound = expect(case, starts, q, 150, 4)
    dec = torch.empty((3, 4, 8, 128), dtype=torch.float16, device="cuda")
    dev = [from_bits(x, "f16").cuda() for x in (q, case["k"], case["v"])]
    pk.pa_decode_window(dec, dev[0].view(3, 4, 8, 128), dev[1], dev[2],
                        torch.from_numpy(case["tables"]).cuda(),
                        torch.from_numpy(case["ctx"]).cuda(), 150, 4, case["scale"],
                        pk.new_workspace(3, 8, 2, 128))
    ref.check(out, dec.double().cpu().view(12, 8, 128), 2 * bound)


def test_captured_on_another_stream_and_two_graphs_of_one_workspace():
    mix = [(300, 900), (1, 64), (70, 70)]
    case, starts, q = setup(mix, 32, 8, 64, 16, "bf16", 100, 4, 4)
    want, _ = run(case, starts, q, 100, 4)
    got, _ = run(case, starts, q, 100, 4, stream=torch.cuda.Stream())
    assert torch.equal(got, want)
    dev = [from_bits(x, "bf16").cuda() for x in (q, case["k"], case["v"])]
    tab, cl = torch.from_numpy(case["tables"]).cuda(), torch.from_numpy(case["ctx"]).cuda()
    sd = torch.from_numpy(starts).cuda()
    ws = pk.new_prefill_workspace()
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g in graphs:
        with torch.cuda.graph(g):
            pk.pa_prefill_window(got, *dev, tab, cl, sd, 100, 4, case["scale"], ws)
    for g in graphs + graphs[::-1]:
        got.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)


def test_captured_with_more_items_than_ctas():
    """CTAs that draw items from the workspace's counter, replayed: two graphs in turn on one
    workspace, behind a decode whose launch they overlap, then new chunk lengths."""
    mix = [(1500, 1600), (3, 64), (700, 700), (0, 9), (64, 1000)]
    case, starts, q = setup(mix, 32, 8, 128, 16, "bf16", 150, 4, 4, drop=False)
    want, st = run(case, starts, q, 150, 4)
    assert st == 0
    ref.check(want, *expect(case, starts, q, 150, 4))
    dev = [from_bits(x, "bf16").cuda() for x in (q, case["k"], case["v"])]
    tab, cl = torch.from_numpy(case["tables"]).cuda(), torch.from_numpy(case["ctx"]).cuda()
    sd = torch.from_numpy(starts).cuda()
    ws, dws = pk.new_prefill_workspace(), pk.new_workspace(5, 32, 8, 128)
    got = torch.full_like(want, 7.0)
    dq = torch.randn((5, 32, 128), device="cuda").bfloat16()
    dout = torch.empty_like(dq)
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g in graphs:
        with torch.cuda.graph(g):
            pk.pa_decode_window(dout, dq, dev[1], dev[2], tab, cl, 150, 4, case["scale"], dws)
            pk.pa_prefill_window(got, *dev, tab, cl, sd, 150, 4, case["scale"], ws)
            pk.pa_prefill_window(got, *dev, tab, cl, sd, 150, 4, case["scale"], ws)
    for g in graphs + graphs[::-1]:
        got.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)
    late = np.array([0, 100, 1400, 1400, 1409, 1409], np.int32)     # other chunks, same graph
    sd.copy_(torch.from_numpy(late))
    got.fill_(7.0)
    graphs[0].replay()
    torch.cuda.synchronize()
    again, st = run(case, late, q, 150, 4)
    # (sequence 3 had no new tokens before, so its rows are poisoned: NaN, compared as bits)
    assert torch.equal(got.view(torch.int16), again.view(torch.int16))
    ref.check(got[:1400], *(x[:1400] for x in expect(case, late, q, 150, 4)))


def test_output_that_is_only_16_byte_aligned():
    case, starts, q = setup([(300, 900), (5, 5)], 8, 2, 64, 16, "f16", 100, 4, 6)
    want, _ = run(case, starts, q, 100, 4)
    dev = [from_bits(x, "f16").cuda() for x in (q, case["k"], case["v"])]
    buf = torch.full((want.numel() + 8,), 7.0, dtype=torch.float16, device="cuda")
    out = buf[8:].view(want.shape)
    assert out.data_ptr() % 32 == 16
    pk.pa_prefill_window(out, *dev, torch.from_numpy(case["tables"]).cuda(),
                         torch.from_numpy(case["ctx"]).cuda(), torch.from_numpy(starts).cuda(),
                         100, 4, case["scale"], pk.new_prefill_workspace())
    assert torch.equal(out, want) and bool((buf[:8] == 7).all())


def test_bad_inputs_are_reported():
    case, starts, q = setup([(40, 200), (50, 300)], 4, 2, 64, 16, "f16", 60, 4, 2, drop=False)
    good, st = run(case, starts, q, 60, 4)
    assert st == 0
    bad = starts.copy()
    bad[2] = 1000                                    # past total_q: that sequence is empty
    out, st = run(case, bad, q, 60, 4)
    assert st == pk.DEV_BAD_QUERY
    assert torch.equal(out[:40], good[:40]) and bool((out[40:] == 7).all())
    bad[1:] = [-5, 90]
    assert run(case, bad, q, 60, 4)[1] == pk.DEV_BAD_QUERY
    t = dict(case, tables=case["tables"].copy())
    t["tables"][1, 3] = case["N"]                    # behind every window
    assert run(t, starts, q, 60, 4)[1] == 0
    t["tables"][1, 17] = -2
    out, st = run(t, starts, q, 60, 4)
    assert st == pk.DEV_BAD_BLOCK_ID and torch.equal(out[:40], good[:40])
    assert run(dict(case, ctx=np.array([200, -4], np.int32)), starts, q, 60, 4)[1] == \
        pk.DEV_BAD_CONTEXT_LEN


def test_refusals():
    case, starts, q = setup([(4, 20), (5, 30)], 4, 2, 64, 16, "f16", 60, 4, 2)
    dev = [from_bits(x, "f16").cuda() for x in (q, q, case["k"], case["v"])]
    ok = dev + [torch.from_numpy(case["tables"]).cuda(), torch.from_numpy(case["ctx"]).cuda(),
                torch.from_numpy(starts).cuda(), 60, 4, 0.1, pk.new_prefill_workspace()]
    pk.pa_prefill_window(*ok)
    for at, bad in ((1, dev[1][:-1]), (6, ok[6][:-1]), (6, ok[6].long()), (7, 0), (8, -1),
                    (9, float("nan")), (10, ok[10][:100]), (2, dev[2].cpu()),
                    (2, dev[2].bfloat16()), (7, 60.0)):
        args = list(ok)
        args[at] = bad
        with pytest.raises(pk.PagedKVError):
            pk.pa_prefill_window(*args)
