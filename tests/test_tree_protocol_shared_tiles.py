"""A model of what the tensor-core tree attention kernel keeps in its two Q tiles, on the CPU.

The kernel (csrc/tree_tc.cu) gives its two streams of softmax warps two tiles of query rows in shared
memory.  Before a run both streams write their share of the run's Q (both tiles for more than 128 rows,
else tile 0), a named barrier tells the MMA warp, and the S products read the tiles until the last of
them has finished.  In a run of one tile the streams exchange their (max, sum) through tile 1.  Loaders,
barriers and clock are those of the models beside it; checked here, under random timing, is that

* every S product finds its run's Q in its tile when it is issued and when it has finished, and
* both streams find this run's (max, sum) when they read the exchange.

Planted mistakes must be caught: a stream's last P.V that may be issued before the other stream's last S (the
stream then goes on to the next run's Q while that S still reads), and an exchange without a barrier
behind its reads.
"""

import random

import pytest

from test_tree_protocol_model import SLOTS, TreeSim, loader, random_runs


class TileSim(TreeSim):
    def __init__(self, seed, last_pv_first=False, unguarded_exchange=False):
        super().__init__(seed)
        self.last_pv_first, self.unguarded_exchange = last_pv_first, unguarded_exchange
        self.q = [[None, None], [None, None]]     # [tile][the stream that writes this half of its rows]
        self.exchange = [None, None]              # (max, sum) of each stream, over tile 1

    def write_q(self, tile, stream, run):
        self.q[tile][stream] = run
        if tile == 1:
            self.exchange = [None, None]

    def check_q(self, tile, run):
        if self.q[tile] != [run, run]:
            raise AssertionError(f"S of run {run} reads a Q tile that holds {self.q[tile]}")

    def issue_s(self, tile, run):
        self.check_q(tile, run)
        self.mma(4)
        self.seq += 1
        self.events.append((max(self.mma_free_at, self.now) + 1, self.seq, lambda: self.check_q(tile, run)))


def mma(sim, runs):
    ring = base = 0
    for r, (nt, two) in enumerate(runs):
        yield "q"
        per = 4 if two else 2
        steps = per * nt
        ns = no = 0
        k_at = lambda i: ring + 2 * (i // per)  # noqa: E731
        use = lambda i: base + (i >> 1)  # noqa: E731
        landed = lambda g: sim.full[g % SLOTS].passed(g // SLOTS)  # noqa: E731
        while no < steps:
            w, u = ns & 1, use(ns)
            if ns < steps and ns < no + 4 and landed(k_at(ns)) and (ns < 4 or sim.o_done[w][u & 1].passed((u >> 1) - 1)):
                sim.issue_s(w if two else 0, r)
                sim.commit(sim.s_full[w][u & 1])
                if ns % per == per - 1:
                    sim.commit(sim.empty[k_at(ns) % SLOTS])
                ns += 1
            w, u = no & 1, use(no)
            # a stream's last P.V tells it that the run's Q is no longer read
            if no < ns and (sim.last_pv_first or no + 2 != steps or ns == steps) and \
                    sim.p_full[w][u & 1].passed(u >> 1) and landed(k_at(no) + 1):
                sim.mma(sim.rng.choice([5, 40]))
                if no % per == per - 1:
                    sim.commit(sim.empty[(k_at(no) + 1) % SLOTS])
                sim.commit(sim.o_done[w][u & 1])
                no += 1
            yield
            yield from sim.pause(60 if sim.rng.random() < 0.1 else 1)   # the warp may be held up
        ring += 2 * nt
        base += steps // 2


def softmax(sim, runs, w):
    use = 0
    for r, (nt, two) in enumerate(runs):
        for tile in range(2 if two else 1):
            yield from sim.pause(2)
            sim.write_q(tile, w, r)
        yield "q"
        for _ in range(2 * nt if two else nt):
            while not sim.s_full[w][use & 1].passed(use >> 1):
                yield
            yield from sim.pause(8)
            sim.p_full[w][use & 1].arrive()
            use += 1
        while not sim.o_done[w][(use - 1) & 1].passed((use - 1) >> 1):
            yield
        if not two:
            sim.exchange[w] = r
            yield "exchange"
            yield from sim.pause(4)
            if sim.exchange != [r, r]:
                raise AssertionError("the exchanged (max, sum) was overwritten before it was read")
            if not sim.unguarded_exchange:
                yield "exchange"
        yield from sim.pause(6 if sim.rng.random() < 0.5 else 0)   # epilogue; a warp without rows has none


def run(runs, seed, max_steps=200000, **planted):
    sim = TileSim(seed, **planted)
    roles = {"load k": loader(sim, runs, 0), "load v": loader(sim, runs, 1), "mma": mma(sim, runs), "s0": softmax(sim, runs, 0), "s1": softmax(sim, runs, 1)}
    waiting, finished = {}, set()
    for _ in range(max_steps):
        if len(finished) == len(roles):
            return True
        order = list(roles)
        sim.rng.shuffle(order)
        for name in order:
            if name in finished or name in waiting:
                continue
            for _ in range(sim.rng.randint(1, 3)):
                try:
                    got = next(roles[name])
                except StopIteration:
                    finished.add(name)
                    break
                if got is not None:
                    waiting[name] = got
                    break
        for barrier, members in (("q", {"mma", "s0", "s1"}), ("exchange", {"s0", "s1"})):
            if {n for n, b in waiting.items() if b == barrier} == members:
                for n in members:
                    del waiting[n]
        sim.now += 1          # step by step: a role may get far while one product runs
        for event in sorted((e for e in sim.events if e[0] <= sim.now), key=lambda e: e[:2]):
            sim.events.remove(event)
            event[2]()
    return False


def test_every_run_completes_on_its_own_q_and_exchange():
    for seed in range(400):
        assert run(random_runs(random.Random(seed)), seed), f"deadlock, seed {seed}"


@pytest.mark.parametrize("planted,what", [(dict(last_pv_first=True), "S of run"), (dict(unguarded_exchange=True), "exchanged")])
def test_planted_mistakes_are_caught(planted, what):
    caught = 0
    for seed in range(400):
        try:
            assert run(random_runs(random.Random(seed)), seed, **planted)
        except AssertionError as e:
            assert what in str(e)
            caught += 1
    assert caught > 0
