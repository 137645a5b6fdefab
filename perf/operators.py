"""The bounded-cache operators, as a serving program calls them, beside their plain forms.

Four kinds of case:
  decode   attention of each sequence's newest token(s) over a paged cache with a sliding
           window and a few first tokens that stay visible (``pa_decode_window``, and
           ``pa_decode_window_e4m3_bs`` over 8-bit pools with per-(block, kv head) scales);
  prefill  the same attention for prompt chunks of ragged lengths (``pa_prefill_window``);
  compact  the kept tokens of a sequence moved to the front of its pages
           (``pa_compact_tokens``, ``pa_compact_tokens_e4m3_bs``).

``run`` computes the plain form in 32 bits with elementary torch operations, or, where
``own`` is true, makes the library's calls.
"""
import math
import random

import torch

own = False

F8_MAX = 448.0
# A serving program keeps one scratch buffer for all its attention calls.
SCRATCH_BYTES = 32 << 20


def listed():
    return [
        # one interactive chat far into its context: the latency of a single token
        dict(name="decode_one", kind="decode", dtype="f16", pool="16", B=1, q_len=1, Hq=32, Hkv=8,
             D=128, bs=16, ctx_lo=20001, ctx_hi=20001, window=1024, sinks=4, dropped=True,
             lens_seed=1),
        # a serving batch of a 70B-shape model (64/8 heads, 1000 to 8000 tokens each)
        dict(name="decode_70b", kind="decode", dtype="bf16", pool="16", B=32, q_len=1, Hq=64,
             Hkv=8, D=128, bs=16, ctx_lo=1000, ctx_hi=8000, window=4096, sinks=4, dropped=True,
             lens_seed=2),
        # the same batch verifying 4 speculated tokens per sequence, an odd window
        dict(name="decode_spec4", kind="decode", dtype="bf16", pool="16", B=32, q_len=4, Hq=64,
             Hkv=8, D=128, bs=16, ctx_lo=1000, ctx_hi=8000, window=1001, sinks=5, dropped=False,
             lens_seed=2),
        # a large batch with a heavy-tailed length mix, small pages
        dict(name="decode_heavytail", kind="decode", dtype="f16", pool="16", B=256, q_len=1,
             Hq=32, Hkv=8, D=128, bs=8, ctx_lo=16, ctx_hi=32768, window=2048, sinks=16,
             dropped=True, lens_seed=4),
        # an 8B-shape batch over 8-bit pages
        dict(name="decode_e4m3", kind="decode", dtype="bf16", pool="e4m3_bs", B=64, q_len=1,
             Hq=32, Hkv=8, D=128, bs=16, ctx_lo=128, ctx_hi=2048, window=1024, sinks=4,
             dropped=False, lens_seed=5),
        # the last few tokens of a prompt whose head is already cached; a small model
        dict(name="prefill_tail", kind="prefill", dtype="f16", B=1, q_lo=37, q_hi=37, Hq=4, Hkv=4,
             D=64, bs=16, past_lo=1500, past_hi=1500, window=256, sinks=4, lens_seed=6),
        # one step of chunked prefill: ragged chunks of many requests at different depths
        dict(name="prefill_mixed", kind="prefill", dtype="f16", B=24, q_lo=1, q_hi=512, Hq=32,
             Hkv=8, D=128, bs=16, past_lo=0, past_hi=4000, window=1024, sinks=4, lens_seed=7),
        # two whole prompts, shorter than the window in part (plain causal attention there)
        dict(name="prefill_8b", kind="prefill", dtype="f16", B=2, q_lo=2000, q_hi=4000, Hq=32,
             Hkv=8, D=128, bs=16, past_lo=0, past_hi=0, window=2048, sinks=4, lens_seed=8),
        # one long prompt of a 70B-shape model: the largest case
        dict(name="prefill_70b", kind="prefill", dtype="bf16", B=1, q_lo=8000, q_hi=8000, Hq=64,
             Hkv=8, D=128, bs=16, past_lo=0, past_hi=0, window=4096, sinks=4, lens_seed=9),
        # one request, one layer: first tokens and the most recent ones kept, in place
        dict(name="compact_one", kind="compact", pool="bf16", L=1, B=1, Hkv=8, D=128, bs=16,
             ctx_lo=1300, ctx_hi=1300, keep=513, per_layer=False, per_head=False, in_place=True,
             lens_seed=10),
        # a batch, several layers, each layer and kv head with a selection of its own, into
        # fresh pages (the sequences' pages are shared with forks)
        dict(name="compact_heads", kind="compact", pool="bf16", L=4, B=16, Hkv=8, D=128, bs=16,
             ctx_lo=2000, ctx_hi=6000, keep=1024, per_layer=True, per_head=True, in_place=False,
             lens_seed=11),
        # 8-bit pages with block scales: the kept rows are quantised anew for their new block
        dict(name="compact_e4m3", kind="compact", pool="e4m3_bs", L=2, B=16, Hkv=8, D=128, bs=16,
             ctx_lo=1000, ctx_hi=3000, keep=700, per_layer=True, per_head=True, in_place=False,
             lens_seed=12),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["decode", "decode", "prefill", "prefill", "compact"])
    bs = rng.choice([1, 8, 16, 16, 32])
    D = rng.choice([64, 128, 128])
    c = dict(kind=kind, D=D, bs=bs, lens_seed=rng.randrange(1 << 20))
    if kind == "compact":
        hi = _log(rng, 40, 6000)
        B = _log(rng, 1, 32)
        L = _log(rng, 1, 8)
        while L * B * hi > 250_000:
            L, B = max(1, L // 2), max(1, B - 1)
        c.update(pool=rng.choice(["f16", "bf16", "e4m3", "e4m3_bs"]), L=L, B=B,
                 Hkv=rng.choice([1, 2, 4, 8]), ctx_lo=max(1, hi // 3), ctx_hi=hi,
                 keep=_log(rng, 1, max(1, hi // 2)), per_layer=rng.random() < 0.5,
                 per_head=rng.random() < 0.5, in_place=rng.random() < 0.5)
        return c
    Hq, Hkv = rng.choice([(4, 4), (32, 8), (64, 8), (16, 1), (20, 4), (6, 2)])
    c.update(Hq=Hq, Hkv=Hkv, dtype=rng.choice(["f16", "bf16"]), window=_log(rng, 8, 4096),
             sinks=rng.choice([0, 1, 4, 5, 16, 33]))
    if kind == "decode":
        pool = rng.choice(["16", "16", "e4m3_bs"])
        hi = _log(rng, 16, 32768)
        B = _log(rng, 1, 256)
        while B * hi > 260_000 or B * min(hi, c["window"] + 50) * Hkv > 4_000_000:
            B = max(1, B * 3 // 4)
            if B == 1:
                break
        rows = 16 if pool == "e4m3_bs" else 64
        c.update(pool=pool, B=B, q_len=min(rng.choice([1, 1, 1, 2, 3, 4, 8]), rows * Hkv // Hq),
                 ctx_lo=rng.choice([0, hi // 8, hi]), ctx_hi=hi, dropped=rng.random() < 0.5)
    else:
        q_hi = _log(rng, 1, 2048)
        past = rng.choice([0, _log(rng, 1, 8000)])
        B = _log(rng, 1, 16)
        while B * q_hi * Hq * min(q_hi + past, q_hi + c["window"] + 40) > 800_000_000 and B > 1:
            B -= 1
        c.update(B=B, q_lo=rng.choice([0, 1, q_hi]), q_hi=q_hi, past_lo=past // 4, past_hi=past)
    return c


def _lens(c, lo, hi, salt=0):
    """Whole numbers of a batch, from the case alone: spread over the logarithm where the
    range spans more than a factor of ten, the largest one always among them."""
    r = random.Random(c["lens_seed"] * 7 + salt)
    if hi > 10 * max(1, lo):
        v = [_log(r, max(1, lo), hi) if lo or r.random() > 0.15 else 0 for _ in range(c["B"])]
    else:
        v = [r.randint(lo, hi) for _ in range(c["B"])]
    v[r.randrange(c["B"])] = hi
    return v


def _shapes(c):
    """(new tokens, context lengths) of an attention case."""
    if c["kind"] == "decode":
        return [c["q_len"]] * c["B"], _lens(c, c["ctx_lo"], c["ctx_hi"])
    q = _lens(c, c["q_lo"], c["q_hi"])
    past = _lens(c, c["past_lo"], c["past_hi"], 1)
    return q, [a + b for a, b in zip(q, past)]


def _first_visible(c, q, ctx):
    """The first position that the oldest new token's window reaches."""
    return max(0, min(ctx, ctx - q - c["window"] + 1))


def _visible(c, q, ctx):
    """(distinct positions that some new token sees, (new token, position) pairs)."""
    pairs, w, s = 0, c["window"], c["sinks"]
    for p in range(max(0, ctx - q), ctx):
        pairs += min(p + 1, w) + min(s, max(0, p + 1 - w))
    w0 = _first_visible(c, q, ctx)
    return ctx - w0 + min(s, w0), pairs


def _keep_lens(c):
    ctx = _lens(c, c["ctx_lo"], c["ctx_hi"])
    return ctx, [min(c["keep"], n // 2 + 1) for n in ctx]


def work(case):
    c = case
    if c["kind"] == "compact":
        _, n = _keep_lens(c)
        rows = sum(n) * c["L"] * c["Hkv"] * 2
        return {"bytes": 2 * rows * c["D"] * (1 if "e4m3" in c["pool"] else 2) + 4 * sum(n),
                "flops": 0}
    q, ctx = _shapes(c)
    seen = [_visible(c, a, b) for a, b in zip(q, ctx)]
    elem = 1 if c.get("pool") == "e4m3_bs" else 2
    return {"bytes": sum(t for t, _ in seen) * c["Hkv"] * c["D"] * 2 * elem
            + 2 * sum(q) * c["Hq"] * c["D"] * 2,
            "flops": 4 * sum(p for _, p in seen) * c["Hq"] * c["D"]}


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _block_scale(amax):
    """The power of two s with s / 16 < amax / 448 <= s / 8; 1 for a row of zeros."""
    m, e = torch.frexp(amax / F8_MAX)
    c = torch.where(m == 0.5, e - 1, e) + 3
    return torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), c.clamp(-126, 127)),
                       torch.ones_like(amax))


def _to_e4m3(x, scale):
    return (x / scale).clamp(-F8_MAX, F8_MAX).to(torch.float8_e4m3fn)


def _pools(shape, pool, g):
    """K and V pools (and the block scales of 8-bit ones), as a server's appends left them."""
    kv, sc = [], []
    for _ in range(2):
        x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
        if pool == "e4m3_bs":
            # [..., block, head, token, dim]: a block's first token sets its scale
            s = _block_scale(x[..., 0, :].abs().amax(-1))
            kv.append(_to_e4m3(x, s[..., None, None]).view(torch.uint8))
            sc.append(s)
        elif pool == "e4m3":
            kv.append(_to_e4m3(x, 1.0 / 64).view(torch.uint8))
        else:
            kv.append(x.to(torch.bfloat16 if pool == "bf16" else torch.float16))
    return kv, sc


def _tables(c, lens, holes, g):
    """Block tables over a shuffled pool; the entries in holes[s] are pages given back."""
    bs = c["bs"]
    need = [[i for i in range(-(-n // bs)) if i not in h] for n, h in zip(lens, holes)]
    blocks = sum(len(x) for x in need)
    order = torch.randperm(blocks + 3, generator=g, device="cuda").to(torch.int32)
    width = max(1, max(-(-n // bs) for n in lens))
    flat = [r * width + i for r, x in enumerate(need) for i in x]
    t = torch.full((len(lens) * width,), -1, dtype=torch.int32, device="cuda")
    t[torch.tensor(flat, dtype=torch.int64, device="cuda")] = order[:blocks]
    return t.view(len(lens), width), blocks + 3


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    if c["kind"] == "compact":
        return _prepare_compact(c, g)
    q, ctx = _shapes(c)
    holes = [()] * c["B"]
    if c.get("dropped"):        # pages wholly behind the window were given back
        bs = c["bs"]
        holes = [range(-(-c["sinks"] // bs), _first_visible(c, a, b) // bs)
                 for a, b in zip(q, ctx)]
    tables, blocks = _tables(c, ctx, holes, g)
    dtype = torch.bfloat16 if c["dtype"] == "bf16" else torch.float16
    kv, sc = _pools((blocks, c["Hkv"], c["bs"], c["D"]),
                    "e4m3_bs" if c.get("pool") == "e4m3_bs" else c["dtype"], g)
    total = sum(q)
    qs = torch.randn((total, c["Hq"], c["D"]), generator=g, device="cuda").to(dtype)
    starts = [0]
    for a in q:
        starts.append(starts[-1] + a)
    if c["kind"] == "decode":
        qs = qs.view(c["B"], c["q_len"], c["Hq"], c["D"])
        if c["q_len"] == 1:
            qs = qs[:, 0]
    return dict(case=c, q=qs, out=torch.empty_like(qs), k=kv[0], v=kv[1], scales=sc,
                tables=tables, ctx=torch.tensor(ctx, dtype=torch.int32, device="cuda"),
                starts=torch.tensor(starts, dtype=torch.int32, device="cuda"),
                scale=1.0 / math.sqrt(c["D"]), q_max=max(q), ctx_max=max(ctx),
                scratch=torch.empty(SCRATCH_BYTES, dtype=torch.uint8, device="cuda"))


def _prepare_compact(c, g):
    ctx, n = _keep_lens(c)
    L, B, H, kmax = c["L"], c["B"], c["Hkv"], max(n)
    bs = c["bs"]
    tables, blocks = _tables(c, ctx, [()] * B, g)
    dst_w = -(-kmax // bs)
    if c["in_place"]:
        dst, total = tables[:, :dst_w].contiguous(), blocks
    else:                       # the pages are shared with a fork: the result takes fresh ones
        fresh = torch.arange(blocks, blocks + B * dst_w, dtype=torch.int32, device="cuda")
        dst, total = fresh.view(B, dst_w), blocks + B * dst_w
    # keep[l][s][h]: ascending positions.  In place: the first tokens and then a choice from
    # the later part; else a choice from the whole context.
    kl, kh = (L if c["per_layer"] else 1), (H if c["per_head"] else 1)
    cl = torch.tensor(ctx, device="cuda").view(1, B, 1, 1)
    nl = torch.tensor(n, device="cuda").view(1, B, 1, 1)
    pos = torch.arange(max(ctx), device="cuda").view(1, 1, 1, -1)
    score = torch.rand((kl, B, kh, max(ctx)), generator=g, device="cuda")
    if c["in_place"]:
        first = torch.minimum(torch.full_like(nl, 4), nl)
        score = torch.where(pos < first, 2.0, torch.where(pos < nl, -1.0, score))
    score = torch.where(pos < cl, score, torch.full_like(score, -2.0))
    top = score.argsort(dim=-1, descending=True)[..., :kmax]
    i = torch.arange(kmax, device="cuda").view(1, 1, 1, -1)
    top = torch.where(i < nl, top, torch.full_like(top, 1 << 30)).sort(dim=-1).values
    keep = torch.where(i < nl, top, torch.zeros_like(top)).to(torch.int32).contiguous()
    kv, sc = _pools((L, total, H, bs, c["D"]), c["pool"], g)
    return dict(case=c, k=kv[0], v=kv[1], scales=sc, tables=tables, dst=dst, keep=keep,
                ctx=torch.tensor(ctx, dtype=torch.int32, device="cuda"),
                n=torch.tensor(n, dtype=torch.int32, device="cuda"))


def run(state):
    kind = state["case"]["kind"]
    if own:
        return _own_compact(state) if kind == "compact" else _own_attend(state)
    return _plain_compact(state) if kind == "compact" else _plain_attend(state)


def _own_attend(s):
    from paged_kv_cache_348_b200 import pagedkv as pk

    c = s["case"]
    if c["kind"] == "prefill":
        pk.pa_prefill_window(s["out"], s["q"], s["k"], s["v"], s["tables"], s["ctx"],
                             s["starts"], c["window"], c["sinks"], s["scale"], s["scratch"])
    elif c["pool"] == "e4m3_bs":
        pk.pa_decode_window_e4m3_bs(s["out"], s["q"], s["k"], s["v"], s["scales"][0],
                                    s["scales"][1], s["tables"], s["ctx"], c["window"],
                                    c["sinks"], s["scale"], s["scratch"])
    else:
        pk.pa_decode_window(s["out"], s["q"], s["k"], s["v"], s["tables"], s["ctx"],
                            c["window"], c["sinks"], s["scale"], s["scratch"])
    return s["out"]


def _own_compact(s):
    from paged_kv_cache_348_b200 import pagedkv as pk

    k, v = list(s["k"].unbind(0)), list(s["v"].unbind(0))
    if s["scales"]:
        ks, vs = s["scales"]
        pk.pa_compact_tokens_e4m3_bs(k, v, list(ks.unbind(0)), list(vs.unbind(0)), s["tables"],
                                     s["dst"], s["ctx"], s["keep"], s["n"])
    else:
        pk.pa_compact_tokens(k, v, s["tables"], s["dst"], s["ctx"], s["keep"], s["n"])
    return _pool_values(s)


def _pool_values(s):
    """The pools after a compaction: 8-bit ones as the E4M3 numbers that they hold."""
    if "e4m3" in s["case"]["pool"]:
        return [s["k"].view(torch.float8_e4m3fn), s["v"].view(torch.float8_e4m3fn), *s["scales"]]
    return [s["k"], s["v"]]


def _rows(pool, scales, tables, pos, bs):
    """Cached rows at positions pos[s][j] in 32 bits: [sequences, kv heads, j, D]."""
    blk = tables.long().gather(1, (pos // bs).clamp(0, tables.shape[1] - 1)).clamp(min=0)
    x = pool[blk, :, pos % bs]
    if scales is None:
        return x.float().transpose(1, 2)
    x = x.view(torch.float8_e4m3fn).float()
    return (x * scales[blk][..., None]).transpose(1, 2)


def _plain_attend(s):
    c, ctx, starts = s["case"], s["ctx"].long(), s["starts"].long()
    B, Hkv, G, D, bs = c["B"], c["Hkv"], c["Hq"] // c["Hkv"], c["D"], c["bs"]
    W, S, QL = c["window"], c["sinks"], s["q_max"]
    flat = s["q"].reshape(-1, c["Hq"], D)
    if not flat.shape[0]:
        return s["q"].clone()
    n = (starts[1:] - starts[:-1])[:, None]                      # new tokens of each sequence
    j = torch.arange(QL, device="cuda")[None]
    at = (starts[:-1, None] + j).clamp(max=flat.shape[0] - 1)    # rows of the padded batch
    q = flat[at].float().view(B, QL, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * QL, D)
    p = torch.where(j < n, ctx[:, None] - n + j, -1)             # positions of the new tokens
    # the positions that some new token sees: the first ones, and the window's
    w0 = (ctx - n[:, 0] - W + 1).clamp(min=0)[:, None]
    span = min(s["ctx_max"], QL + W - 1)
    first = torch.arange(S, device="cuda")[None].expand(B, S)
    t = torch.cat([torch.where(first < w0, first, 1 << 40),
                   w0 + torch.arange(span, device="cuda")[None]], 1)
    valid = t < ctx[:, None]
    t = torch.where(valid, t, 0)
    sc = s["scales"] or [None, None]
    k = _rows(s["k"], sc[0], s["tables"], t, bs)
    v = _rows(s["v"], sc[1], s["tables"], t, bs)
    v = v * valid[:, None, :, None]
    x = torch.matmul(q, k.transpose(2, 3)).mul_(s["scale"]).view(B, Hkv, G, QL, -1)
    see = (t[:, None] <= p[..., None]) & valid[:, None]
    see &= (t[:, None] > p[..., None] - W) | (t[:, None] < S)
    x.masked_fill_(~see[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    x.sub_(torch.where(m > -math.inf, m, 0.0)).exp_()
    z = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(B, Hkv, G * QL, -1), v).view(B, Hkv, G, QL, D)
    o = torch.where(z > 0, o / z, 0.0).permute(0, 3, 1, 2, 4).reshape(B, QL, c["Hq"], D)
    row = torch.arange(flat.shape[0], device="cuda")
    b = torch.searchsorted(starts[1:].contiguous(), row, right=True)
    return o[b, row - starts[b]].to(flat.dtype).view(s["q"].shape)


def _plain_compact(s):
    c, bs = s["case"], s["case"]["bs"]
    shape = (c["L"], c["B"], c["Hkv"], s["keep"].shape[-1])
    keep = s["keep"].long().expand(shape)
    # row i of the result; the padding past a sequence's count repeats its row 0
    i = torch.arange(shape[3], device="cuda").expand(shape)
    i = torch.where(i < s["n"].view(1, -1, 1, 1), i, 0)
    t = keep.gather(3, i)
    layer = torch.arange(shape[0], device="cuda").view(-1, 1, 1, 1)
    seq = torch.arange(shape[1], device="cuda").view(1, -1, 1, 1)
    head = torch.arange(shape[2], device="cuda").view(1, 1, -1, 1)
    src = s["tables"].long()[seq, t // bs]
    dst = s["dst"].long()[seq, i // bs]
    if s["scales"]:
        _requantise(s["k"], s["scales"][0], layer, head, src, t % bs, dst, i, bs)
        _requantise(s["v"], s["scales"][1], layer, head, src, t % bs, dst, i, bs)
    else:
        s["k"][layer, dst, head, i % bs] = s["k"][layer, src, head, t % bs]
        s["v"][layer, dst, head, i % bs] = s["v"][layer, src, head, t % bs]
    return _pool_values(s)


def _requantise(pool, scales, layer, head, src, off, dst, i, bs):
    x = pool.view(torch.float8_e4m3fn)[layer, src, head, off].float()
    x = x * scales[layer, src, head][..., None]
    new = _block_scale(x.abs().amax(-1)).gather(3, i - i % bs)   # set by a block's first row
    pool[layer, dst, head, i % bs] = _to_e4m3(x, new[..., None]).view(torch.uint8)
    scales[layer, dst, head] = new


def exact(case, seed):
    """Attention from its definition in 64 bits, one sequence and kv head at a time."""
    c = dict(case)
    s = prepare(c, seed)
    if c["kind"] == "compact":
        return _exact_compact(c, s)
    G, W, S, bs = c["Hq"] // c["Hkv"], c["window"], c["sinks"], c["bs"]
    q = s["q"].reshape(-1, c["Hq"], c["D"]).double()
    out = torch.zeros_like(q)
    starts, ctxs, tables = s["starts"].tolist(), s["ctx"].tolist(), s["tables"].tolist()
    for b in range(c["B"]):
        n, ctx = starts[b + 1] - starts[b], ctxs[b]
        if n == 0 or ctx == 0:
            continue
        held = [i for i in range(-(-ctx // bs)) if tables[b][i] >= 0]
        blk = torch.tensor([tables[b][i] for i in held], device="cuda")
        t = (torch.tensor(held, device="cuda")[:, None] * bs
             + torch.arange(bs, device="cuda")).reshape(-1)
        inside = t < ctx
        t = t[inside]
        for h in range(c["Hkv"]):
            kv = []
            for i, pool in enumerate((s["k"], s["v"])):
                x = pool[blk, h]
                if s["scales"]:
                    x = x.view(torch.float8_e4m3fn).double()
                    x = x * s["scales"][i][blk, h].double()[:, None, None]
                kv.append(x.double().reshape(-1, c["D"])[inside])
            for r0 in range(0, n, 1024):
                r1 = min(n, r0 + 1024)
                p = torch.arange(ctx - n + r0, ctx - n + r1, device="cuda")[:, None]
                see = (t <= p) & ((t > p - W) | (t < S))
                for g in range(h * G, (h + 1) * G):
                    rows = q[starts[b] + r0:starts[b] + r1, g]
                    x = (rows @ kv[0].T) * s["scale"]
                    a = torch.where(see, x, torch.full_like(x, -math.inf))
                    top = a.amax(1, keepdim=True).clamp(min=-1e300)
                    e = torch.exp(a - top)
                    z = e.sum(1, keepdim=True)
                    got = (e @ kv[1]) / torch.where(z > 0, z, torch.ones_like(z))
                    out[starts[b] + r0:starts[b] + r1, g] = got
    return out.view(s["q"].shape)


def _exact_compact(c, s):
    """The moved rows one list at a time; 8-bit rows rounded to the E4M3 numbers' grid (steps
    of 2^(e-3) in [2^e, 2^(e+1)), e at least -6) in 64 bits."""
    bs, scales = c["bs"], [x.double() for x in s["scales"]]
    eight = "e4m3" in c["pool"]
    pools = [(x.view(torch.float8_e4m3fn) if eight else x).double() for x in (s["k"], s["v"])]
    for i in range(2):
        for b, n in enumerate(s["n"].tolist()):
            at = torch.arange(n, device="cuda")
            dst, slot = s["dst"][b, at // bs].long(), at % bs
            for layer in range(c["L"]):
                for h in range(c["Hkv"]):
                    t = s["keep"][min(layer, s["keep"].shape[0] - 1), b,
                                  min(h, s["keep"].shape[2] - 1), :n].long()
                    src = s["tables"][b, t // bs].long()
                    x = pools[i][layer, src, h, t % bs]
                    if scales:
                        x = x * scales[i][layer, src, h][:, None]
                        top = x[::bs].abs().amax(1)
                        new = torch.exp2(torch.ceil(torch.log2(top / F8_MAX)) + 3)
                        new = torch.where(top > 0, new, torch.ones_like(new))
                        scales[i][layer, dst[::bs], h] = new
                        y = x / new[at // bs][:, None]
                        e = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6)))
                        step = torch.exp2(e - 3)
                        x = (torch.round(y / step) * step).clamp(-F8_MAX, F8_MAX)
                    pools[i][layer, dst, h, slot] = x
    return [*pools, *scales]
