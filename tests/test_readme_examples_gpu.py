"""The README's verification and eviction, run as printed, on sequences that share blocks with others."""

import os
import re

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")
HQ, HKV, D, B, NB = 8, 2, 64, 16, 96


@pytest.fixture(scope="module")
def pa():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    from paged_kv_cache_382_b200 import build

    build.build()
    from paged_kv_cache_382_b200 import pa as binding

    return binding


def blocks():
    with open(README) as f:
        code = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    return {name: next(c for c in code if key in c) for name, key in
            (("tables", "def tables"), ("verify", "tree_decode("), ("evict", "select_tokens("))}


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Pools:
    """Pools and a block manager; every token's K and V as they were written."""

    def __init__(self, pa):
        self.pa, self.rng = pa, np.random.default_rng(4)
        self.bm = pa.NativeBlockManager(NB, B, free_order=self.rng.permutation(NB))
        self.k = torch.full((NB, HKV, B, D), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.v = self.k.clone()
        self.kept = {}

    def write(self, seq, n):
        slots, copies, _ = self.bm.append(seq, n)
        if copies:
            self.pa.copy_blocks(self.k, self.v, torch.tensor(copies, dtype=torch.int64, device="cuda"))
        k, v = (torch.from_numpy(self.rng.standard_normal((n, HKV, D))).to(torch.bfloat16).cuda() for _ in range(2))
        self.pa.reshape_and_cache(k, v, self.k, self.v, torch.from_numpy(np.ascontiguousarray(slots)).cuda())
        old = self.kept.get(seq, (k[:0], v[:0]))
        self.kept[seq] = (torch.cat([old[0], k]), torch.cat([old[1], v]))

    def rows(self, seq, h):
        table, n = np.array([self.bm.block_table(seq)]), self.bm.num_tokens(seq)
        return [oracle.gather_kv(f64(x), table[0], n, h) for x in (self.k, self.v)]

    def holds(self, seq, positions=None):
        """Whether the sequence's blocks hold its tokens at `positions` ([kv head] lists; None: all of them)."""
        for h in range(HKV):
            want = slice(None) if positions is None else positions[h]
            for got, x in zip(self.rows(seq, h), self.kept[seq]):
                if not np.array_equal(got, f64(x[:, h])[want]):
                    return False
        return True


def test_verification_as_printed(pa):
    p = Pools(pa)
    parents = [[-1] + [i // 2 for i in range(69)], [-1, 0, 0, 2, 3]]      # more than 64 nodes, and fewer
    prefix_lens, paths, seq_ids = [45, 30], [[0, 1, 3, 7, 15], [0, 2, 3]], [0, 1]
    for s in seq_ids:
        p.bm.add(s)
        p.write(s, prefix_lens[s])
        p.write(s, len(parents[s]))
    for s in seq_ids:           # others hold the same blocks, drafted tokens and all
        p.bm.fork(s, 10 + s)
        p.kept[10 + s] = p.kept[s]
    n = [len(x) for x in parents]
    names = dict(pa=pa, torch=torch, bm=p.bm, seq_ids=seq_ids, parents=parents, d=D, k_cache=p.k, v_cache=p.v,
                 context_lens=i32([a + b for a, b in zip(prefix_lens, n)]), query_start=i32([0, n[0], sum(n)]), prefix_lens=prefix_lens,
                 new_lens=[a + len(b) for a, b in zip(prefix_lens, paths)], prefix_lens_dev=i32(prefix_lens),
                 accepted_positions=i32([[[a + x for x in b] + [0] * (5 - len(b))] for a, b in zip(prefix_lens, paths)]),
                 accepted_counts=i32([len(b) for b in paths]),
                 q=torch.randn(sum(n), HQ, D, device="cuda").to(torch.bfloat16))
    names["out"] = torch.empty_like(names["q"], dtype=torch.float32)
    code = blocks()
    exec(code["tables"] + code["verify"], names)
    torch.cuda.synchronize()
    for s in seq_ids:
        keep = list(range(prefix_lens[s])) + [prefix_lens[s] + x for x in paths[s]]
        assert p.bm.num_tokens(s) == len(keep)
        assert p.holds(s, [keep] * HKV) and p.holds(10 + s)
    q, out, at = f64(names["q"]), f64(names["out"]), 0
    for s in seq_ids:
        for i in range(n[s]):
            seen, j = [], i
            while j >= 0:
                seen.append(prefix_lens[s] + j)
                j = parents[s][j]
            seen = list(range(prefix_lens[s])) + seen
            for h in range(HQ):
                k, v = (f64(x[:, h * HKV // HQ])[seen] for x in p.kept[s])
                assert np.abs(out[at + i, h] - oracle.decode_attention_one(q[at + i, h], k, v, D ** -0.5)).max() <= 2e-3
        at += n[s]


def test_eviction_as_printed(pa):
    p = Pools(pa)
    lens, budgets, seq_ids = [300, 90, 200], [100, 128, 199], [0, 1, 2]
    for s in seq_ids:
        p.bm.add(s)
        p.write(s, lens[s])
    for s in (0, 1):
        p.bm.fork(s, 10 + s)
        p.kept[10 + s] = p.kept[s]
    stride = 320
    totals = torch.rand(3, HKV, stride, device="cuda")
    before = totals.clone()
    names = dict(pa=pa, torch=torch, bm=p.bm, seq_ids=seq_ids, d=D, k_cache=p.k, v_cache=p.v, lens=lens, budgets=budgets,
                 context_lens=i32(lens), budgets_dev=i32(budgets), lens_before=i32([n - 1 for n in lens]), totals=totals,
                 keep=torch.full((3, HKV, 199), -1, dtype=torch.int32, device="cuda"), kept_lens=i32([0, 0, 0]),
                 q=torch.randn(3, HQ, D, device="cuda").to(torch.bfloat16))
    names["out"] = torch.empty_like(names["q"])
    k64, table = f64(p.k), [p.bm.block_table(s) for s in seq_ids]
    code = blocks()
    exec(code["tables"] + code["evict"], names)
    torch.cuda.synchronize()
    keep = names["keep"].cpu().numpy()
    exact = oracle.attention_weights(f64(names["q"]), k64, [np.array(t) for t in table], lens, D ** -0.5)
    for s in seq_ids:
        n = min(lens[s], budgets[s])
        assert p.bm.num_tokens(s) == n
        rows = [keep[s, h, :n].tolist() for h in range(HKV)]
        for h in range(HKV):
            old = f64(before[s, h, :lens[s]])
            old[-1] = 0.0
            total = old + exact[s][h]
            assert rows[h] == sorted(rows[h]) and rows[h][-min(64, n):] == list(range(lens[s] - min(64, n), lens[s]))
            # nothing dropped beats anything kept by more than the totals' error
            out = sorted(set(range(lens[s] - 64)) - set(rows[h]))
            if out:
                assert total[out].max() <= total[rows[h][:-64]].min() + 1e-4
            assert np.abs(f64(totals[s, h, :n]) - total[rows[h]]).max() <= 1e-4
        assert p.holds(s, rows)
    assert p.holds(10) and p.holds(11)
