"""The prefix cache never serves a block whose slots hold something else (CPU).

Every test keeps what each physical slot holds: a value that stands for a token's K and V, which depend on
the token and on all before it.  The writes, block copies and moves that the block manager asks for are
applied to these slots, and every position of every sequence has to hold its own value, the positions that
an append found in the cache among them.
"""

import numpy as np
import pytest


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_382_b200 import build

    build.build()
    from paged_kv_cache_382_b200 import pa as binding

    return binding


class Cache:
    """A block manager with prefix caching and the contents of its slots."""

    def __init__(self, pa, num_blocks, block_size, free_order=None):
        self.pa, self.B = pa, block_size
        self.bm = pa.NativeBlockManager(num_blocks, block_size, free_order=free_order, prefix_cache=True)
        self.slots = np.zeros(num_blocks * block_size, dtype=np.int64)   # 0: nothing
        self.seqs = {}          # id -> the values of its tokens
        self.known = {}         # id -> its token ids, None once an eviction made them unknown
        self.unique = -1

    def add(self, s):
        self.bm.add(s)
        self.seqs[s], self.known[s] = [], []

    def fork(self, s, child):
        self.bm.fork(s, child)
        self.seqs[child] = list(self.seqs[s])
        self.known[child] = None if self.known[s] is None else list(self.known[s])

    def free(self, s):
        self.bm.free(s)
        del self.seqs[s], self.known[s]

    def copy(self, pairs):
        old = self.slots.copy()
        for src, dst in pairs:
            self.slots[dst * self.B:(dst + 1) * self.B] = old[src * self.B:(src + 1) * self.B]

    def chain(self, ids):
        return hash(tuple(int(x) for x in ids)) % (1 << 60) + 1

    def value(self, s, token):
        """Of a token appended to s: by the ids before it where they are all known, else of its own."""
        if self.known[s] is None:
            self.unique -= 1
            return self.unique
        self.known[s].append(int(token))
        return self.chain(self.known[s])

    def draft(self, s, tokens):
        """A tree of drafted tokens: values of their own, for no ids say what a node's ancestors are."""
        slots, copies, cached = self.bm.append(s, [-1] * len(tokens))
        assert cached == 0
        self.copy(copies)
        for at, _ in zip(slots, tokens):
            self.unique -= 1
            self.seqs[s].append(self.unique)
            self.slots[at] = self.unique
        self.check()

    def append(self, s, tokens):
        slots, copies, cached = self.bm.append(s, tokens)
        self.copy(copies)
        for at, token in zip(slots, tokens):
            v = self.value(s, token)
            self.seqs[s].append(v)
            if at >= 0:
                self.slots[at] = v
        self.check()
        return cached

    def compact(self, names, unchanged, keeps, ids=None):
        """Sequence names[k] keeps its first unchanged[k] tokens and the positions keeps[k] behind them; ids: a
        list of the kept ones' token ids for each sequence, or None."""
        src = {s: self.bm.block_table(s) for s in names}
        copies = self.bm.compact(names, unchanged, [u + len(k) for u, k in zip(unchanged, keeps)],
                                 None if ids is None else [int(x) for row in ids for x in row])
        self.copy(copies)
        old = self.slots.copy()
        for i, (s, u, keep) in enumerate(zip(names, unchanged, keeps)):
            dst = self.bm.block_table(s)
            for j, p in enumerate(keep):
                self.slots[dst[(u + j) // self.B] * self.B + (u + j) % self.B] = old[src[s][p // self.B] * self.B + p % self.B]
            self.seqs[s] = self.seqs[s][:u] + [self.seqs[s][p] for p in keep]
            if ids is None and keep:
                self.known[s] = None
            elif self.known[s] is not None:
                self.known[s] = self.known[s][:u] + ([] if ids is None else [int(x) for x in ids[i]])
        self.check()

    def check(self):
        for s, values in self.seqs.items():
            table = self.bm.block_table(s)
            held = [int(self.slots[table[p // self.B] * self.B + p % self.B]) for p in range(len(values))]
            assert held == values, f"sequence {s} does not hold its tokens"


@pytest.mark.parametrize("lets_go", ["free", "copy on write"])
def test_cut_inside_a_shared_cached_block_then_the_sharer_lets_go(pa, lets_go):
    c = Cache(pa, 32, 4)
    c.add(1)
    c.append(1, range(1, 9))
    c.fork(1, 2)
    c.compact([1], [6], [[]])
    if lets_go == "free":
        c.free(2)
    else:
        c.compact([2], [6], [[]])
        c.append(2, [50])            # sequence 2 moves to a block of its own
    c.append(1, [70, 80])            # in place
    c.add(3)
    assert c.append(3, range(1, 9)) == 4
    c.add(4)
    assert c.append(4, [1, 2, 3, 4, 5, 6, 70, 80]) == 8


def test_two_forks_cut_in_one_call_then_appended_to(pa):
    c = Cache(pa, 32, 4)
    c.add(1)
    c.append(1, range(1, 9))
    c.fork(1, 2)
    c.compact([1, 2], [6, 6], [[], []])
    c.append(1, [70, 80])
    c.append(2, [90, 91])
    c.add(3)
    assert c.append(3, range(1, 9)) == 4


@pytest.mark.parametrize("seed", range(12))
def test_random_appends_forks_cuts_evictions_and_frees(pa, seed):
    rng = np.random.default_rng(seed)
    NB, B = 48, 4
    c, nxt = Cache(pa, NB, B, rng.permutation(NB)), 0
    for _ in range(250):
        op, names = rng.integers(0, 7), list(c.seqs)
        if op == 0 or not names:
            c.add(nxt)
            c.append(nxt, [1, 2, 3, 4, 5, 6, 7, 8][: rng.integers(1, 9)] if c.bm.num_free > 4 else [])
            nxt += 1
        elif op <= 2:
            s = int(rng.choice(names))
            if c.bm.num_free > 4:
                # few ids: the same blocks come up again and again
                c.append(s, rng.integers(1, 3, size=rng.integers(1, 10)))
        elif op == 3:
            c.fork(int(rng.choice(names)), nxt)
            nxt += 1
        elif op == 4:
            c.free(int(rng.choice(names)))
        else:
            some = [int(x) for x in rng.permutation(names)[: rng.integers(1, 4)]]
            u = [int(rng.integers(0, len(c.seqs[s]) + 1)) for s in some]
            cut = op == 5
            keeps = [[] if cut else sorted(int(p) for p in rng.choice(np.arange(x, len(c.seqs[s])), rng.integers(0, len(c.seqs[s]) - x + 1),
                                                                      replace=False)) for s, x in zip(some, u)]
            if c.bm.num_free > sum(-(-(x + len(k)) // B) for x, k in zip(u, keeps)):
                c.compact(some, u, keeps)
    assert nxt > 20


def test_drafted_trees_do_not_enter_the_cache(pa):
    """Two requests draft trees of several blocks behind the same prefix; neither finds the other's nodes, nor does a
    request whose prompt runs on with the drafted tokens, during the verification or after it."""
    c = Cache(pa, 64, 4)
    for s in (1, 2):
        c.add(s)
        assert c.append(s, range(1, 11)) == (0 if s == 1 else 8)
        c.draft(s, range(20, 33))
    c.add(3)
    assert c.append(3, list(range(1, 11)) + list(range(20, 33))) == 8
    # the accepted path, by its ids: its values are those of the chain
    names, paths = [1, 2], [[20, 22, 25], [21]]
    accepted = {s: [10 + t - 20 for t in p] for s, p in zip(names, paths)}
    for s, p in zip(names, paths):
        for k, at in enumerate(accepted[s]):
            v = c.chain(list(range(1, 11)) + p[: k + 1])
            table = c.bm.block_table(s)
            c.seqs[s][at] = v
            c.slots[table[at // 4] * 4 + at % 4] = v
    c.compact(names, [10, 10], [accepted[s] for s in names], ids=paths)
    c.append(1, [40, 41, 42])
    c.append(2, [40])
    c.add(4)
    assert c.append(4, list(range(1, 11)) + [20, 22, 25, 40, 41, 42]) == 16
    c.add(5)
    assert c.append(5, list(range(1, 11)) + [21, 40]) == 12
    c.draft(5, range(9))
    c.compact([5], [12], [[]])               # nothing accepted
    c.append(5, [50, 51, 52, 53])
    c.add(6)
    assert c.append(6, list(range(1, 11)) + [21, 40, 50, 51, 52, 53]) == 16


def test_blocks_behind_a_draft_are_not_cached(pa):
    c = Cache(pa, 64, 4)
    for s in (1, 2):
        c.add(s)
        c.append(s, [1, 2, 3])
        c.draft(s, [7])
        c.known[s] = None                    # what follows depends on the node
        assert c.append(s, [5, 6, 7, 8]) == 0
    assert not set(c.bm.block_table(1)) & set(c.bm.block_table(2))
