"""The block manager's bounded-cache calls (drop_window, compact) against a plain model of the
tables and counts, and against the definition of what a window sees.  CPU only."""
from __future__ import annotations

import numpy as np
import pytest

from paged_kv_cache_348_b200 import build as pbuild
from paged_kv_cache_348_b200.block_manager import BlockManager, PoolExhausted, plan_cascade_tables


@pytest.fixture(scope="module", autouse=True)
def _library():
    pbuild.build()


class Model:
    """Tables, lengths and the free queue, straight from the description in the header."""

    def __init__(self, n, bs):
        self.n, self.bs, self.free, self.t, self.len, self.next = n, bs, list(range(n)), {}, {}, 0
        self.gone = {}

    def ref(self, b):
        return sum(x == b for t in self.t.values() for x in t)

    def give_back(self, old):
        """Blocks of `old` (just removed from a table) that nobody holds any more."""
        for b in old:
            if b >= 0 and self.ref(b) == 0 and b not in self.free:
                self.free.append(b)

    def allocate(self, tokens):
        nb = -(-tokens // self.bs)
        self.t[self.next] = [self.free.pop(0) for _ in range(nb)]
        self.len[self.next] = tokens
        self.next += 1
        return self.next - 1

    def fork(self, s):
        self.t[self.next], self.len[self.next] = list(self.t[s]), self.len[s]
        self.next += 1
        return self.next - 1

    def append(self, s):
        lb = self.len[s] // self.bs
        if lb == len(self.t[s]):
            self.t[s].append(self.free.pop(0))
        elif self.ref(self.t[s][lb]) > 1:
            self.t[s][lb] = self.free.pop(0)
        self.len[s] += 1

    def release(self, s):
        self.give_back(self.t.pop(s))
        del self.len[s]

    def drop_window(self, s, window, sinks):
        n = 0
        for i, b in enumerate(self.t[s]):
            held = range(i * self.bs, min((i + 1) * self.bs, self.len[s]))
            full = (i + 1) * self.bs <= self.len[s]
            seen = any(t < sinks or t >= self.len[s] - window for t in held)
            if b >= 0 and full and not seen:
                self.t[s][i] = -1
                self.give_back([b])
                n += 1
        return n

    def compact(self, sids, lens):
        own = {s: [b if b >= 0 and self.ref(b) == 1 else None
                   for b in self.t[s][:-(-n // self.bs)]] for s, n in zip(sids, lens)}
        if sum(b is None for t in own.values() for b in t) > len(self.free):
            raise MemoryError
        new = {s: [self.free.pop(0) if b is None else b for b in own[s]] for s in sids}
        for s, n in zip(sids, lens):
            old = self.t[s]
            self.t[s], self.len[s] = new[s], n
            self.give_back(old)
        return [new[s] for s in sids]


def check(m, r):
    for s in r.t:
        assert m.table(s) == r.t[s] and m.context_len(s) == r.len[s]
    assert m.free_blocks == len(r.free)
    for b in range(r.n):
        assert m.refcount(b) == r.ref(b)


@pytest.mark.parametrize("seed", range(12))
def test_random_histories_match_the_model(seed):
    rng = np.random.default_rng(seed)
    bs = int(rng.choice([1, 4, 8]))
    m, r = BlockManager(60, bs), Model(60, bs)
    for _ in range(120):
        op, live = rng.integers(0, 7), list(r.t)
        s = int(rng.choice(live)) if live else None
        if op == 0 or s is None:
            n = int(rng.integers(0, 9 * bs))
            if -(-n // bs) <= len(r.free):
                assert m.allocate(n) == r.allocate(n)
        elif op == 1:
            assert m.fork(s) == r.fork(s)
        elif op == 2 and len(r.free) > 1:
            r.append(s)
            m.append_token(s)
        elif op == 3:
            m.release(s)
            r.release(s)
        elif op == 4:
            w, k = int(rng.integers(1, 4 * bs)), int(rng.integers(0, 3 * bs))
            assert m.drop_window(s, w, k) == r.drop_window(s, w, k)
        elif op == 5:
            some = [int(x) for x in rng.permutation(live)[:3]]
            lens = [int(rng.integers(0, r.len[x] + 1)) for x in some]
            try:
                want = r.compact(some, lens)
            except MemoryError:
                with pytest.raises(PoolExhausted):
                    m.compact(some, lens)
            else:
                got = m.compact(some, lens, fill=-3)
                for row, t in zip(got, want):
                    assert list(row[:len(t)]) == t and all(x == -3 for x in row[len(t):])
        elif op == 6:
            # out and in again: the same holes, fresh blocks from the front of the queue
            held = [b for b in r.t[s] if b >= 0]
            assert list(m.swap_out(s)) == held
            holes = [b < 0 for b in r.t[s]]
            old, r.t[s] = r.t[s], []
            r.give_back(old)
            if len(held) > len(r.free):           # its shared blocks stayed with the others
                with pytest.raises(PoolExhausted):
                    m.swap_in(s)
                m.release(s)
                r.release(s)
            else:
                assert list(m.swap_in(s)) == r.free[:len(held)]
                r.t[s] = [-1 if h else r.free.pop(0) for h in holes]
        check(m, r)


def test_drop_window_keeps_every_page_that_a_later_token_sees():
    for bs in (1, 8, 16):
        for length in (0, 1, 15, 16, 17, 100, 333):
            for window in (1, 2, 16, 17, 90, 1000, 1 << 40):
                for sinks in (0, 1, 16, 20, 1 << 40):
                    m = BlockManager(400, bs)
                    s = m.allocate(length)
                    m.drop_window(s, window, sinks)
                    t = m.table(s)
                    for i, b in enumerate(t):
                        seen = any(x < sinks or x > p - window
                                   for x in range(i * bs, min((i + 1) * bs, length))
                                   for p in (length - 1, length))
                        last = (i + 1) * bs > length          # still filling
                        assert (b >= 0) == (seen or last), (bs, length, window, sinks, i)


def test_refusals_change_nothing():
    m = BlockManager(12, 4)
    a = m.allocate(30)
    b = m.fork(a)
    before = (m.table(a), m.table(b), m.free_blocks)
    for args in ((99, 4, 0), (a, 0, 0), (a, 4, -1)):
        with pytest.raises(ValueError):
            m.drop_window(*args)
    for sids, lens in (([a], [31]), ([a], [-1]), ([99], [3]), ([a, a], [3, 3])):
        with pytest.raises(ValueError):
            m.compact(sids, lens)
    with pytest.raises(ValueError):
        m.compact([a], [30], width=2)
    with pytest.raises(PoolExhausted):
        m.compact([a, b], [30, 30])               # both would need 8 fresh blocks, 4 are free
    assert (m.table(a), m.table(b), m.free_blocks) == before
    m.swap_out(a)
    with pytest.raises(ValueError):
        m.drop_window(a, 4, 0)
    with pytest.raises(ValueError):
        m.compact([a], [3])


def test_tables_with_pages_gone_are_refused_where_they_cannot_work():
    m = BlockManager(40, 4)
    a = m.allocate(40)
    b = m.fork(a)
    assert m.drop_window(a, 6, 0) == 8
    assert m._L.pa_bm_num_blocks_of(m._h, a) == 2 and len(m.table(a)) == 10
    with pytest.raises(ValueError):
        m.slot_of(a, 3)
    assert m.slot_of(a, 39) == m.table(a)[9] * 4 + 3
    with pytest.raises(ValueError):
        m.plan_cascade([a, b], 4)
    with pytest.raises(ValueError):
        plan_cascade_tables(m.block_tables([a, b]), m.context_lens([a, b]), 4, 4)
    m.plan_cascade([b], 4)


def test_tail_waste_counts_held_pages_only():
    m = BlockManager(40, 4)
    a = m.allocate(38)
    assert m.tail_waste([a]) == 2 / 40
    m.drop_window(a, 6, 0)                        # 32 positions and their pages gone
    assert m.tail_waste([a]) == 2 / 8
