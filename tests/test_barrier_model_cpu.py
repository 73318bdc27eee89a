"""The forward kernels' barriers, as a model on the CPU.

A wait on an mbarrier names a phase by its parity alone, so it passes as well
when the phase before last is the completed one.  The model runs the roles of a
CTA (producer, the two issuers, the two softmax warpgroups) in random
interleavings, with copies that land in any order, and fails where a wait
passes on another phase than the one it means, where a product reads a tile that is not
there, or where a copy overwrites one that is still read.  The ring's slots are
read from the kernels' sources.
"""

import os
import random
import re

import pytest

from exact_tiled_attention_08_gb300 import build


class Barrier:
    def __init__(self):
        self.pending, self.copies, self.phase = 1, 0, 0

    def step(self):
        if self.pending == 0 and self.copies == 0:
            self.phase += 1
            self.pending = 1

    def arrive(self):
        assert self.pending, "more arrivals than the phase takes"
        self.pending -= 1
        self.step()

    def expect(self):
        self.copies += 1
        self.arrive()

    def land(self):
        self.copies -= 1
        self.step()


def wait(barrier, use):
    """Waits for phase `use` (counted from 0) by its parity."""
    while barrier.phase & 1 == use & 1:
        yield
    assert barrier.phase == use + 1, ("a wait passed early", barrier.phase, use)


def run(items, slots, dual, seed):
    """`items`: key blocks of tile 0 and of tile 1 of each item (a pair of row
    tiles, or one).  `slots`: of K and of V tiles, or one number for a ring that
    takes both in turn; `dual`: a score buffer per tile."""
    rng = random.Random(seed)
    shared = isinstance(slots, int)
    rings = [slots] * 2 if shared else slots
    full, empty = [[Barrier() for _ in range(slots if shared else sum(slots))] for _ in range(2)]
    s_full, s_free, p_full, pv_done = [[Barrier(), Barrier()] for _ in range(4)]
    q_full, q_empty = Barrier(), Barrier()
    copies, products = [], ([], [])  # products complete in the order of their issue
    tile, used = [None] * len(full), [None] * len(full)

    def place(kv, g):
        """Slot and use of block g's K (kv = 0) or V tile."""
        f = 2 * g + kv if shared else g
        return (0 if shared else kv * rings[0]) + f % rings[kv], f // rings[kv]

    def blocks():
        g = 0
        for n0, n1 in items:
            for j in range(max(n0, n1)):
                yield g, j, [t for t, n in enumerate((n0, n1)) if j < n], j == max(n0, n1) - 1
                g += 1

    def producer():
        def load(kv, g):
            s, u = place(kv, g)
            if u:
                yield from wait(empty[s], u - 1)
            assert used[s] is None, ("a tile still in use is overwritten", kv, g)
            full[s].expect()
            tile[s], used[s] = None, (kv, g)

            def land():
                tile[s] = kv, g
                full[s].land()

            copies.append(land)
            yield

        q = 0
        for g, j, _, _ in blocks():
            yield from load(0, g)
            yield from load(1, g)
            if j == 0:
                if q:
                    yield from wait(q_empty, q - 1)
                q_full.expect()
                copies.append(q_full.land)
                q += 1

    def product(kv, g, barrier):
        def read():
            assert tile[place(kv, g)[0]] == (kv, g), ("a product reads another tile", kv, g)

        products[kv].extend([read, barrier.arrive])

    def release(kv, g):
        def done():
            used[place(kv, g)[0]] = None
            empty[place(kv, g)[0]].arrive()

        products[kv].append(done)

    def s_issuer():
        q, uses = 0, [0, 0]
        for g, j, tiles, last in blocks():
            if j == 0:
                yield from wait(q_full, q)
                q += 1
            s, u = place(0, g)
            yield from wait(full[s], u)
            for t in tiles:
                b = t if dual else 0
                if uses[b]:
                    yield from wait(s_free[b], uses[b] - 1)
                product(0, g, s_full[t])
                uses[b] += 1
                yield
            release(0, g)
            if last:
                products[0].append(q_empty.arrive)
            yield

    def pv_issuer():
        uses = [0, 0]
        for g, _, tiles, _ in blocks():
            s, u = place(1, g)
            yield from wait(full[s], u)
            for t in tiles:
                yield from wait(p_full[t], uses[t])
                product(1, g, pv_done[t])
                uses[t] += 1
                yield
            release(1, g)
            yield

    def softmax(t):
        uses = 0
        for n in (x[t] for x in items):
            for j in range(n):
                yield from wait(s_full[t], uses)
                s_free[t if dual else 0].arrive()
                yield
                if j:
                    yield from wait(pv_done[t], uses - 1)
                p_full[t].arrive()
                uses += 1
                yield
            if n:
                yield from wait(pv_done[t], uses - 1)

    roles = {f.__name__: f() for f in (producer, s_issuer, pv_issuer)}
    roles.update({"softmax 0": softmax(0), "softmax 1": softmax(1)})
    speed = {name: rng.choice([1, 1, 5, 20]) for name in [*roles, "copies", 0, 1]}
    in_order = rng.random()
    steps = 0
    while roles or copies or products[0] or products[1]:
        steps += 1
        assert steps < 20000, "no role can go on"
        names = [*roles, *(["copies"] if copies else []), *(i for i in (0, 1) if products[i])]
        name = rng.choices(names, [speed[n] for n in names])[0]
        if name == "copies":
            copies.pop(0 if rng.random() < in_order else rng.randrange(len(copies)))()
        elif name in (0, 1):
            products[name].pop(0)()
        else:
            try:
                next(roles[name])
            except StopIteration:
                del roles[name]


def ring(source, d):
    """Slots of the K/V ring at head dimension d."""
    text = open(os.path.join(build.CSRC_DIR, source)).read()
    slots = re.search(r"kSlots = .*?\(?D == 128\)? \? (\d+) : (\d+)", text)
    slots = int(slots.group(1 if d == 128 else 2))
    return ((slots + 1) // 2, slots // 2) if "kKSlots = (kSlots + 1) / 2, kVSlots = kSlots / 2" in text else slots


# items of two row tiles, of one, of both kinds (a last round, a head's last rows), causal ones
ITEMS = {
    "pairs": lambda n, r: [(n, n)],
    "single": lambda n, r: [(n, 0)],
    "mixed": lambda n, r: [(m, m * r.randint(0, 1)) for m in (n, r.randint(1, 6), r.randint(1, 6), r.randint(1, 20))],
    "causal": lambda n, r: [(n | 1, (n | 1) + 1), (5, 0), (1, 2), (4, 0)],
}


@pytest.mark.parametrize("items", ITEMS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("source", ["fa_fwd.cuh", "fa_cross_fwd.cuh"])
def test_no_wait_passes_early(source, d, items):
    slots = ring(source, d)
    for seed in range(250):
        r = random.Random(seed)
        run(ITEMS[items](r.choice([1, 2, 4, 9, 30]), r), slots, d == 64, seed)
