"""A model of the tensor-core tree attention kernel's barrier protocol, on the CPU.

The kernel (csrc/tree_tc.cu) runs two loader warps (K, V), an MMA-issuing warp
and two streams of softmax warps per CTA; the loaders run ahead over the CTA's
runs, the others meet at a named barrier before each run.  As for the prefill
kernel's model, whose barriers and clock this one uses: every run must complete
under random timing, and no parity wait may look at a barrier that is two phases
on.  The token masks' ring, which has no "free" barrier of its own, is checked
too: no mask may be overwritten before the stream that needs it has read it, and
O may be scaled only while none of the stream's P.V runs.  Planted mistakes must
be caught: a single mask instead of a ring, and an S issued before the P.V that
reads the same buffer has finished.
"""

import random

import pytest

from test_prefill_protocol_model import Barrier, Sim

SLOTS, MASKS = 5, 4


class TreeSim(Sim):
    def __init__(self, seed, masks=MASKS, early_s=False):
        super().__init__(seed)
        self.masks, self.early_s = masks, early_s
        self.full = [Barrier(f"full[{i}]") for i in range(SLOTS)]
        self.empty = [Barrier(f"empty[{i}]") for i in range(SLOTS)]
        self.masked = [Barrier(f"masked[{i}]") for i in range(masks)]
        self.mask = [None] * masks
        pair = lambda n: [[Barrier(f"{n}[{w}][{b}]") for b in range(2)] for w in range(2)]  # noqa: E731
        self.s_full, self.p_full, self.o_done = pair("s_full"), pair("p_full"), pair("o_done")
        self.reading = [[0, 0], [0, 0]]     # P.V issued and not finished, per stream and buffer

    def finish_pv(self, w, b):
        def done():
            self.reading[w][b] -= 1
            self.o_done[w][b].arrive()
        at = max(self.mma_free_at, self.now) + 1
        self.seq += 1
        self.events.append((at, self.seq, done))


def loader(sim, runs, v):
    ring, tile = v, 0
    for nt, two in runs:
        for _ in range(nt):
            slot = ring % SLOTS
            if ring >= SLOTS:
                while not sim.empty[slot].passed(ring // SLOTS - 1):
                    yield
            yield from sim.pause(2)
            sim.full[slot].arrive(tx=64)
            sim.copy(sim.full[slot], 64)
            if v == 0:
                yield from sim.pause(1)
                sim.mask[tile % sim.masks] = tile
                sim.masked[tile % sim.masks].arrive()
            ring += 2
            tile += 1


def mma(sim, runs):
    ring = base = 0
    for nt, two in runs:
        yield "sync"
        per = 4 if two else 2
        steps = per * nt
        ns = no = 0
        k_at = lambda i: ring + 2 * (i // per)  # noqa: E731
        use = lambda i: base + (i >> 1)  # noqa: E731
        landed = lambda g: sim.full[g % SLOTS].passed(g // SLOTS)  # noqa: E731
        while no < steps:
            w, u = ns & 1, use(ns)
            if ns < steps and ns < no + 4 + sim.early_s and landed(k_at(ns)) and \
                    (ns < 4 or sim.early_s or sim.o_done[w][u & 1].passed((u >> 1) - 1)):
                if sim.reading[w][u & 1]:
                    raise AssertionError("S issued over weights that a P.V still reads")
                sim.mma(4)
                sim.commit(sim.s_full[w][u & 1])
                if ns % per == per - 1:
                    sim.commit(sim.empty[k_at(ns) % SLOTS])
                ns += 1
            w, u = no & 1, use(no)
            if no < ns and sim.p_full[w][u & 1].passed(u >> 1) and landed(k_at(no) + 1):
                sim.mma(5)
                sim.reading[w][u & 1] += 1
                if no % per == per - 1:
                    sim.commit(sim.empty[(k_at(no) + 1) % SLOTS])
                sim.finish_pv(w, u & 1)
                no += 1
            yield
            yield from sim.pause(2)
        ring += 2 * nt
        base += steps // 2


def softmax(sim, runs, w):
    ring = tiles = use = 0
    for nt, two in runs:
        yield "sync"
        for k in range(2 * nt if two else nt):
            j = k >> 1 if two else k
            t = tiles + j
            while not sim.masked[t % sim.masks].passed(t // sim.masks):
                yield
            if sim.mask[t % sim.masks] != t:
                raise AssertionError("a token mask was overwritten before it was read")
            while not sim.s_full[w][use & 1].passed(use >> 1):
                yield
            if sim.rng.random() < 0.3:          # tokens that take no part: V is zeroed
                g = ring + 2 * j + 1
                while not sim.full[g % SLOTS].passed(g // SLOTS):
                    yield
            if k and sim.rng.random() < 0.3:    # O scaled
                while not sim.o_done[w][(use - 1) & 1].passed((use - 1) >> 1):
                    yield
                if any(sim.reading[w]):
                    raise AssertionError("O scaled while a P.V adds to it")
            yield from sim.pause(8)
            sim.p_full[w][use & 1].arrive()
            use += 1
        while not sim.o_done[w][(use - 1) & 1].passed((use - 1) >> 1):
            yield
        ring += 2 * nt
        tiles += nt


def run(runs, seed, max_steps=200000, **planted):
    sim = TreeSim(seed, **planted)
    roles = {"load k": loader(sim, runs, 0), "load v": loader(sim, runs, 1), "mma": mma(sim, runs), "s0": softmax(sim, runs, 0), "s1": softmax(sim, runs, 1)}
    at_sync, finished = set(), set()
    for _ in range(max_steps):
        if len(finished) == len(roles):
            return True
        order = list(roles)
        sim.rng.shuffle(order)
        for name in order:
            if name in finished or name in at_sync:
                continue
            for _ in range(sim.rng.randint(1, 3)):
                try:
                    got = next(roles[name])
                except StopIteration:
                    finished.add(name)
                    break
                if got == "sync":
                    at_sync.add(name)
                    break
        if at_sync == {"mma", "s0", "s1"}:       # the loaders do not take part
            at_sync.clear()
        if sim.events:
            sim.events.sort(key=lambda e: e[:2])
            sim.now = sim.events[0][0]
            while sim.events and sim.events[0][0] <= sim.now:
                sim.events.pop(0)[2]()
        else:
            sim.now += 1
    return False


def random_runs(rng):
    return [(rng.randint(1, 9), rng.random() < 0.5) for _ in range(rng.randint(1, 6))]


def test_protocol_completes_and_no_wait_falls_two_phases_behind():
    for seed in range(400):
        assert run(random_runs(random.Random(seed)), seed), f"deadlock, seed {seed}"


@pytest.mark.parametrize("planted", [dict(masks=1), dict(early_s=True)])
def test_planted_mistakes_are_caught(planted):
    caught = 0
    for seed in range(300):
        try:
            ok = run(random_runs(random.Random(seed)), seed, max_steps=4000, **planted)
        except AssertionError:
            ok = False
        caught += not ok
    assert caught > 0
