"""What a decode workspace holds on entry does not matter: words that look like another call's
arrival counters (a small number above a count, as two neighbouring 32-bit indices make them),
and what calls with other grids left behind."""
from __future__ import annotations

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from paged_kv_cache_348_b200 import inputs
from paged_kv_cache_348_b200 import pagedkv as pk
from tests.helpers import bits, from_bits, make_case

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CTX = [2000, 700, 1500, 333, 64, 1999]


class Calls:
    """Split decodes of one small batch: few and many query rows, plain and windowed."""

    def __init__(self):
        case = make_case(len(CTX), 4, 1, 64, 16, CTX, dtype="f16", seed=7)
        self.kv = [from_bits(case[x], "f16").cuda() for x in ("k", "v")]
        self.tab = torch.from_numpy(case["tables"]).cuda()
        self.ctx = torch.from_numpy(case["ctx"]).cuda()
        self.q = [from_bits(bits(inputs.randn((len(CTX), n, 4, 64), "f16", 7, stream=11)),
                            "f16").cuda() for n in (1, 5)]          # 4 and 20 query rows
        self.ws = pk.new_workspace(len(CTX), 4, 1, 64)

    def __call__(self, wide, window=0):
        out = torch.full_like(self.q[wide], float("nan"))
        if window:
            pk.pa_decode_window(out, self.q[wide], *self.kv, self.tab, self.ctx, window, 4, 0.125,
                                self.ws)
        else:
            pk.pa_decode_multi(out, self.q[wide], *self.kv, self.tab, self.ctx, 0.125, self.ws)
        return out


def scan(first, fill):
    """Calls `first`, `first` + 1, ... of this process, each on a workspace filled for it."""
    c = Calls()
    c.ws.zero_()
    want = [c(0), c(1)]
    words = c.ws[:c.ws.numel() // 8 * 8].view(torch.int64)
    for i in range(3, first):
        c(i % 2)
    bad = []
    for i in range(max(first, 3), max(first, 3) + 300):
        fill(words, i)
        if not torch.equal(c(i % 2), want[i % 2]):
            bad.append(i)
    return bad


def count_words(words, i):
    """Every word a thousand arrivals under the number i."""
    words.fill_((i << 32) | 1000)


def index_words(words, i):
    """0, 1, 2, ... as 32-bit numbers."""
    words.view(torch.int32).copy_(torch.arange(2 * words.numel(), dtype=torch.int32,
                                               device="cuda"))


@pytest.mark.parametrize("fill", ["count_words", "index_words"])
def test_words_that_look_like_counters(fill):
    """In a process of its own, so that the i-th call is known."""
    code = ("from tests import test_gpu_workspace_contents as t\n"
            "bad = t.scan(1, t.%s)\n"
            "print('BAD', len(bad), bad[:10])\n" % fill)
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True,
                       timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    assert "BAD 0 []" in r.stdout, r.stdout[-500:]


def test_calls_with_other_grids_in_turn():
    """Grids of one CTA to all of them on one workspace, which is never cleared: the counters
    of a larger one lie over the partial results of a smaller one."""
    c = Calls()
    kinds = [(w, win) for w in (0, 1) for win in (0, 1, 40, 333, 5000)]
    want = {}
    for kind in kinds:
        c.ws.zero_()
        want[kind] = c(*kind)
    c.ws.fill_(0xFF)
    rng = np.random.default_rng(0)
    for i in rng.integers(0, len(kinds), 200):
        assert torch.equal(c(*kinds[i]), want[kinds[i]]), kinds[i]
    graphs = {}
    for kind in kinds:                               # the same, each kind captured once
        graphs[kind] = (torch.cuda.CUDAGraph(), None)
        torch.cuda.synchronize()
        with torch.cuda.graph(graphs[kind][0]):
            out = c(*kind)
        graphs[kind] = (graphs[kind][0], out)
    for i in rng.integers(0, len(kinds), 200):
        g, out = graphs[kinds[i]]
        out.fill_(float("nan"))
        g.replay()
        assert torch.equal(out, want[kinds[i]]), kinds[i]
