"""A model of chunk attention's ring of K and V tiles, run in many orders on the CPU.

Entry 2 i of the ring is K tile i, entry 2 i + 1 V tile i, entry e uses stage e mod STAGES.  A loading warp
each for K and V, the warps that clean the edge tiles of V, and the warp of each query tile's MMAs take their
steps in any order that the waits allow (those on logits, weights, queries and turns are left out: the model
allows more orders than the kernel).  What it shows: how many V tiles can be loaded and not cleaned, which
barriers of edge tiles that takes, and that what a CTA drains at its end covers every copy in flight when a
wait gave up, and waits for no other phase."""
import os
import random
import re

import pytest

STAGES = 5
SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "decode_kv_cache_03_gb300", "csrc",
                      "kara_chunk.cu")


def mma_program(x, pieces):
    """What the warp of query tile x waits for and gives back, in order: ("full", entry), ("empty", entry)."""
    ops, k0 = [], 0
    for two, n, cnt0 in pieces:
        k_at, v_at = [k0], [k0]   # next K and V tile

        def take(at, kv):
            e = 2 * at[0] + kv
            at[0] += 1
            return [("full", e)], [("empty", e)]

        cnt = (cnt0 if x == 0 else n) if two else (n + 1 - x) // 2
        by, first = (1, 0) if two else (2, x)
        last = first + (cnt - 1) * by
        t = first - by
        while t < n:
            if not two and x == 1 and t >= 0:
                ops += sum(take(v_at, 1), [])
            v_back = []
            if first <= t < n:
                wait, v_back = take(v_at, 1)
                ops += wait
                if two and t + 1 < n:
                    ops.append(("full", 2 * k_at[0]))
                if not (two and t <= last):
                    ops, v_back = ops + v_back, []
            if not two and x == 0 and t >= 0 and t + 1 < n:
                ops += sum(take(v_at, 1), [])
            if not two and x == 1 and t + 1 < n:
                ops += sum(take(k_at, 0), [])
            if t + by < n:
                wait, back = take(k_at, 0)
                ops += wait + back
            ops += v_back
            if not two and x == 0 and t + by + 1 < n:
                ops += sum(take(k_at, 0), [])
            t += by
        if not two and x == 1 and n % 2:
            ops += sum(take(v_at, 1), [])
        assert k_at[0] == v_at[0] == k0 + n
        k0 += n
    return ops, k0


class Ring:
    def __init__(self, pieces, edges, rng):
        self.rng, self.edges = rng, edges
        self.mma = [mma_program(x, pieces)[0] for x in (0, 1)]
        self.tiles = mma_program(0, pieces)[1]
        self.pc, self.issued = [0, 0], [0, 0]
        self.landed, self.clean, self.empty = set(), set(), {}
        self.ne = self.nclean = self.most = 0
        self.edge_no = []   # V tiles that are edge tiles, as issued

    def full(self, e):
        return e in self.clean if e % 2 and self.edges[e // 2] else e in self.landed

    def steps(self):
        """What can happen next."""
        todo = []
        for kv in (0, 1):
            e = 2 * self.issued[kv] + kv
            if self.issued[kv] < self.tiles and (e < STAGES or self.empty.get(e - STAGES) == 2):
                todo.append(("load", e))
            todo += [("land", f) for f in range(kv, e, 2) if f not in self.landed]
        if self.nclean < self.ne and 2 * self.edge_no[self.nclean] + 1 in self.landed:
            todo.append(("clean", 2 * self.edge_no[self.nclean] + 1))
        for x in (0, 1):
            if self.pc[x] < len(self.mma[x]):
                what, e = self.mma[x][self.pc[x]]
                if what == "empty" or self.full(e):
                    todo.append(("mma", x))
        return todo

    def step(self, what, arg):
        if what == "load":
            if arg >= STAGES:
                assert self.full(arg - STAGES)    # nothing is loaded over a tile in flight
            self.issued[arg % 2] += 1
            if arg % 2 and self.edges[arg // 2]:
                self.ne += 1
                self.edge_no.append(arg // 2)
            out = [e for e in range(1, 2 * self.issued[1], 2) if not self.full(e)]
            self.most = max(self.most, len(out))
        elif what == "land":
            self.landed.add(arg)
        elif what == "clean":
            self.clean.add(arg)
            self.nclean += 1
        else:
            op, e = self.mma[arg][self.pc[arg]]
            self.pc[arg] += 1
            if op == "empty":
                self.empty[e] = self.empty.get(e, 0) + 1
                assert self.empty[e] <= 2

    def drained(self, kv, slots):
        """Entries that the warp of K or V waits for at the end: by their stage, by their edge barrier."""
        k, others = self.issued[kv], self.issued[1 - kv]
        full = [2 * (k - d) + kv for d in range(1, min(slots, k) + 1)]
        full = [e for e in full if (e + STAGES) // 2 >= others and not (kv and self.edges[e // 2])]
        return full, [2 * i + 1 for i in self.edge_no[max(0, self.ne - slots):]] if kv else []


def run(seed, slots):
    rng = random.Random(seed)
    pieces = []
    for _ in range(rng.randrange(1, 6)):
        n = rng.choice([1, 1, 2, 3, 4, 9])
        two = rng.random() < 0.4
        pieces.append((two, n, rng.randrange(max(0, n - 2), n + 1)))
    total = sum(n for _, n, _ in pieces)
    share = rng.choice([0.0, 0.5, 1.0])
    r = Ring(pieces, [rng.random() < share for _ in range(total)], rng)
    slow = rng.choice(["clean", "land", "mma", None])     # one that comes last wherever it can
    stop = rng.choice([None, rng.randrange(1, 12 * total + 2)])
    n = 0
    while True:
        todo = r.steps()
        if not todo or n == stop:
            break
        fast = [s for s in todo if s[0] != slow]
        r.step(*rng.choice(fast if fast and rng.random() < 0.95 else todo))
        n += 1
    if stop is None:
        assert r.pc == [len(m) for m in r.mma] and r.issued == [total, total]
    flying = {e for kv in (0, 1) for e in range(kv, 2 * r.issued[kv], 2) if e not in r.landed}
    covered = set()
    for kv in (0, 1):
        full, edge = r.drained(kv, slots)
        for e in full:   # its stage's phase is the last one: nothing has been loaded behind it
            assert (e + STAGES) // 2 >= r.issued[(e + STAGES) % 2]
        for i, e in enumerate(reversed(edge)):
            assert i < slots   # (as many barriers: the next use of this one is not yet)
        covered |= set(full) | set(edge)
    return r.most, flying <= covered


@pytest.fixture(scope="module")
def slots():
    text = open(SOURCE).read()
    assert re.search(r"constexpr int kStages = %d;" % STAGES, text)
    assert "constexpr int kEdges = (kStages - 1) / 2 + 2;" in text
    return (STAGES - 1) // 2 + 2


def test_tiles_in_flight_have_a_barrier_each_and_are_drained(slots):
    most = 0
    for seed in range(4000):
        m, all_covered = run(seed, slots)
        most = max(most, m)
        assert all_covered, seed
    assert most == slots


def test_three_would_not_do(slots):
    assert not all(run(seed, slots - 1)[1] for seed in range(4000))
