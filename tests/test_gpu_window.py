"""pa_decode_window and pa_decode_window_e4m3_bs against the 64-bit definition: masks, odd
sizes, pages given back, what lies outside the window poisoned with NaN, refusals."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
from paged_kv_cache_348_b200 import inputs
from paged_kv_cache_348_b200 import pagedkv as pk
from tests import window_ref as ref
from tests.helpers import NAN_BITS, bits, from_bits, make_case
from tests.test_gpu_fp8_bs import bs_case

pytestmark = pytest.mark.gpu

CTX = [0, 1, 2, 5, 15, 16, 17, 40, 63, 64, 65, 130, 200, 513, 1000, 2047]


def seen_rows(ctx, q_len, window, sinks):
    """Positions of one sequence that some new token sees."""
    pos = torch.arange(max(0, ctx - q_len), ctx)
    if not len(pos):
        return np.zeros(0, bool)
    return ref.visible(pos, torch.arange(ctx), window, sinks).any(0).numpy()


def poison(case, q_len, window, sinks, drop):
    """NaN into every slot that no new token sees; junk into the table entries of blocks
    without a seen slot (drop)."""
    bs = case["bs"]
    used = np.zeros((case["N"], bs), bool)
    for i in range(case["B"]):
        seen = seen_rows(int(case["ctx"][i]), q_len, window, sinks)
        for b0 in range(0, len(seen), bs):
            blk = case["tables"][i][b0 // bs]
            s = seen[b0:b0 + bs]
            used[blk, :len(s)] |= s
            if drop and not s.any():
                case["tables"][i][b0 // bs] = [-1, 1 << 30, -(1 << 31)][(b0 // bs) % 3]
    return ~used


def gathered(case, i, pool):
    """Cached rows of sequence i as double [ctx, Hkv, D] (unreadable blocks as zeros)."""
    ctx, bs = int(case["ctx"][i]), case["bs"]
    out = torch.zeros((-(-ctx // bs) * bs, case["Hkv"], case["D"]), dtype=torch.double)
    for b in range(-(-ctx // bs)):
        blk = int(case["tables"][i][b])
        if 0 <= blk < case["N"]:
            out[b * bs:(b + 1) * bs] = pool[blk].transpose(0, 1)
    return out[:ctx]


def expected(case, q, k, v, window, sinks, u_p):
    """(out, bound) of the whole batch; q double [B, QL, Hq, D], pools double."""
    outs = []
    for i in range(case["B"]):
        ctx, QL = int(case["ctx"][i]), q.shape[1]
        pos = torch.arange(ctx - QL, ctx)
        outs.append(ref.attend(q[i], gathered(case, i, k), gathered(case, i, v), pos, window,
                               sinks, case["scale"], u_p, case["dtype"]))
    return torch.stack([o for o, _ in outs]), torch.stack([b for _, b in outs])


def run16(case, q, window, sinks, stream=None):
    dt = case["dtype"]
    out = torch.full(q.shape, float("nan"), dtype=inputs.torch_dtype(dt), device="cuda")
    ws = pk.new_workspace(case["B"], case["Hq"], case["Hkv"], case["D"])
    ws.fill_(0xFF)
    st = pk.new_status()
    pk.pa_decode_window(out, from_bits(q, dt).cuda(), from_bits(case["k"], dt).cuda(),
                        from_bits(case["v"], dt).cuda(),
                        torch.from_numpy(np.ascontiguousarray(case["tables"])).cuda(),
                        torch.from_numpy(case["ctx"]).cuda(), window, sinks, case["scale"], ws,
                        st, stream)
    torch.cuda.synchronize()
    return out, int(st.item())


def u_p16(dtype, rows):
    """P as the kernels hold it: up to 8 rows two 16-bit parts; the tcgen05 kernel two bf16
    parts or one fp16 part."""
    if dtype == "bf16":
        return 2.0 ** -16
    return 2.0 ** -22 if rows <= 8 else 2.0 ** -11


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D,bs", [(64, 1), (64, 8), (64, 16), (64, 32), (128, 1), (128, 8),
                                  (128, 16), (128, 32)])
@pytest.mark.parametrize("Hq,Hkv,q_len", [(8, 2, 1), (4, 4, 3), (16, 1, 1), (8, 2, 5), (12, 2, 8)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (7, 3), (64, 4), (100, 0), (129, 33)])
def test_shapes(dtype, D, bs, Hq, Hkv, q_len, window, sinks):
    case = make_case(len(CTX), Hq, Hkv, D, bs, CTX, dtype=dtype, seed=D + bs + Hq + q_len,
                     poison=False)
    mask = poison(case, q_len, window, sinks, drop=(window + bs) % 2 == 0)
    for p in ("k", "v"):
        case[p].transpose(0, 2, 1, 3)[mask] = NAN_BITS[dtype]
    q = bits(inputs.randn((case["B"], q_len, Hq, D), dtype, 3, stream=11))
    out, st = run16(case, q, window, sinks)
    assert st == 0
    dbl = {x: from_bits(case[x], dtype).double() for x in ("k", "v")}
    want, bound = expected(case, from_bits(q, dtype).double(), dbl["k"], dbl["v"], window, sinks,
                           u_p16(dtype, Hq // Hkv * q_len))
    ref.check(out, want, bound, "decode_window")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D,bs", [(64, 1), (64, 16), (128, 1), (128, 8), (128, 16), (128, 32)])
@pytest.mark.parametrize("Hq,Hkv,q_len", [(8, 2, 1), (8, 2, 4), (4, 4, 3)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (7, 3), (100, 17)])
def test_e4m3_shapes(dtype, D, bs, Hq, Hkv, q_len, window, sinks):
    case = bs_case(np.array(CTX, np.int32), Hq, Hkv, bs, dtype, seed=D + bs + q_len, q_len=q_len,
                   D=D)
    if q_len == 1:
        case["q"] = case["q"].reshape(case["B"], 1, Hq, D)
    mask = poison(case, q_len, window, sinks, drop=True)
    for p in ("k8", "v8"):
        case[p].transpose(0, 2, 1, 3)[mask] = 0x7F
    for p in ("ks", "vs"):
        case[p][mask.all(1)] = np.nan
    out = torch.full(case["q"].shape, float("nan"), dtype=inputs.torch_dtype(dtype), device="cuda")
    st = pk.new_status()
    pk.pa_decode_window_e4m3_bs(
        out, from_bits(case["q"], dtype).cuda(), torch.from_numpy(case["k8"]).cuda(),
        torch.from_numpy(case["v8"]).cuda(), torch.from_numpy(case["ks"]).cuda(),
        torch.from_numpy(case["vs"]).cuda(),
        torch.from_numpy(np.ascontiguousarray(case["tables"])).cuda(),
        torch.from_numpy(case["ctx"]).cuda(), window, sinks, case["scale"],
        pk.new_workspace(case["B"], Hq, Hkv, D), st)
    assert int(st.item()) == 0
    pools = [(torch.from_numpy(case[a]).view(torch.float8_e4m3fn).double()
              * torch.from_numpy(case[b]).double()[:, :, None, None])
             for a, b in (("k8", "ks"), ("v8", "vs"))]
    # q goes to fp16 exactly (normal values); P times the V scale is held in fp16
    want, bound = expected(case, from_bits(case["q"], dtype).double(), *pools, window, sinks,
                           2.0 ** -11)
    # P V in fp16 also when q and out are bf16: weights below fp16's normal range
    bound = bound + (want != 0) * 2048 * 2.0 ** -24 * 2.0 ** -3
    ref.check(out, want, bound, "decode_window_e4m3_bs")


@pytest.mark.parametrize("q_len,Hq", [(1, 8), (1, 32), (4, 64)])
def test_window_past_the_context_is_pa_decode_multi(q_len, Hq):
    case = make_case(len(CTX), Hq, 8, 128, 16, CTX, dtype="bf16", seed=5)
    q = bits(inputs.randn((case["B"], q_len, Hq, 128), "bf16", 5, stream=11))
    want = torch.empty(q.shape, dtype=torch.bfloat16, device="cuda")
    ws = pk.new_workspace(case["B"], Hq, 8, 128)
    dev = [from_bits(x, "bf16").cuda() for x in (q, case["k"], case["v"])]
    tab, ctx = torch.from_numpy(case["tables"]).cuda(), torch.from_numpy(case["ctx"]).cuda()
    pk.pa_decode_multi(want, *dev, tab, ctx, case["scale"], ws)
    for window, sinks in ((2047, 0), (1 << 40, 9), (1, 2047), (5, 1 << 40)):
        out, st = run16(case, q, window, sinks)
        assert st == 0 and torch.equal(out, want), (window, sinks)


def test_one_token_form_and_block_permutation():
    ctx = [700, 33, 1, 2048, 129, 0, 64, 1500]
    case = make_case(len(ctx), 32, 8, 128, 16, ctx, dtype="f16", seed=9)
    q = bits(inputs.randn((8, 1, 32, 128), "f16", 9, stream=11))
    out, _ = run16(case, q, 333, 4)
    flat, _ = run16(case, np.ascontiguousarray(q[:, 0]), 333, 4)
    assert torch.equal(out[:, 0], flat)
    perm = np.random.default_rng(1).permutation(case["N"])
    moved = dict(case, k=np.empty_like(case["k"]), v=np.empty_like(case["v"]))
    moved["k"][perm], moved["v"][perm] = case["k"], case["v"]
    moved["tables"] = np.where(case["tables"] >= 0, perm[case["tables"].clip(0)], -7).astype(np.int32)
    again, st = run16(moved, q, 333, 4)
    assert st == 0 and torch.equal(out, again)


def test_a_bad_page_in_the_window_is_reported_and_one_behind_it_is_not():
    case = make_case(2, 8, 2, 128, 16, [500, 500], dtype="f16", seed=2)
    q = bits(inputs.randn((2, 1, 8, 128), "f16", 2, stream=11))
    case["tables"][0, 5] = case["N"] + 3          # positions 80..95: behind the window
    assert run16(case, q, 64, 4)[1] == 0
    case["tables"][0, 0] = -1                     # the first tokens
    assert run16(case, q, 64, 0)[1] == 0
    assert run16(case, q, 64, 4)[1] == pk.DEV_BAD_BLOCK_ID
    case["ctx"][1] = 1 << 20                      # beyond the table
    assert run16(case, q, 64, 0)[1] == pk.DEV_BAD_CONTEXT_LEN


def test_captured_and_on_another_stream():
    ctx = [900, 64, 333, 1]
    case = make_case(4, 32, 8, 128, 16, ctx, dtype="bf16", seed=4)
    q = bits(inputs.randn((4, 2, 32, 128), "bf16", 4, stream=11))
    want, _ = run16(case, q, 100, 4)
    s = torch.cuda.Stream()
    out, _ = run16(case, q, 100, 4, stream=s)
    assert torch.equal(out, want)
    dev = [from_bits(x, "bf16").cuda() for x in (q, case["k"], case["v"])]
    tab, cl = torch.from_numpy(case["tables"]).cuda(), torch.from_numpy(case["ctx"]).cuda()
    ws = pk.new_workspace(4, 32, 8, 128)
    got = torch.empty_like(want)
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]        # two graphs, one workspace
    for g in graphs:
        with torch.cuda.graph(g):
            pk.pa_decode_window(got, *dev, tab, cl, 100, 4, case["scale"], ws)
    for g in graphs + graphs:
        got.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)
    cl.copy_(torch.tensor([64, 900, 17, 0], device="cuda"))   # lengths of a later step
    graphs[0].replay()
    case["ctx"] = np.array([64, 900, 17, 0], np.int32)
    assert torch.equal(got, run16(case, q, 100, 4)[0])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("Hq,q_len", [(4, 1), (16, 2)])
@pytest.mark.parametrize("scale", [0.0, -0.2, 2.5])
def test_scales(dtype, Hq, q_len, scale):
    case = make_case(len(CTX), Hq, 1, 128, 16, CTX, dtype=dtype, seed=12, poison=False)
    mask = poison(case, q_len, 60, 4, drop=True)
    for p in ("k", "v"):
        case[p].transpose(0, 2, 1, 3)[mask] = NAN_BITS[dtype]
    case["scale"] = scale
    q = bits(inputs.randn((case["B"], q_len, Hq, 128), dtype, 3, stream=11))
    out, st = run16(case, q, 60, 4)
    assert st == 0
    dbl = {x: from_bits(case[x], dtype).double() for x in ("k", "v")}
    ref.check(out, *expected(case, from_bits(q, dtype).double(), dbl["k"], dbl["v"], 60, 4,
                             u_p16(dtype, Hq * q_len)))


def test_refusals():
    case = make_case(2, 8, 2, 64, 16, [100, 20], dtype="f16", seed=2)
    q = from_bits(case["q"], "f16").cuda()
    ok = [torch.empty_like(q), q, from_bits(case["k"], "f16").cuda(), from_bits(case["v"], "f16").cuda(),
          torch.from_numpy(case["tables"]).cuda(), torch.from_numpy(case["ctx"]).cuda(), 30, 4, 0.1,
          pk.new_workspace(2, 8, 2, 64)]
    pk.pa_decode_window(*ok)
    for at, bad in ((1, q[:1]), (0, ok[0].bfloat16()), (2, ok[2].transpose(1, 2)), (4, ok[4].long()),
                    (5, ok[5][:1]), (6, 0), (6, 3.5), (7, -1), (8, float("inf")),
                    (9, ok[9][:64]), (3, ok[3].cpu())):
        args = list(ok)
        args[at] = bad
        with pytest.raises(pk.PagedKVError):
            pk.pa_decode_window(*args)
    with pytest.raises(pk.PagedKVError):                       # 16-bit pools are not 8-bit ones
        pk.pa_decode_window_e4m3_bs(*ok[:4], ok[2], ok[2], *ok[4:])
