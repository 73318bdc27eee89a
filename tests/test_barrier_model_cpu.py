"""The forward kernels' barriers, as a model on the CPU.

A wait on an mbarrier names a phase by its parity alone, so it passes as well
when the phase before last is the completed one.  The model runs the roles of a
CTA (producer, the two issuers, the two softmax warpgroups) in random
interleavings, with copies that land in any order, and fails where a wait
passes on another phase than the one it means, where a product reads a tile that is not
there, or where a copy overwrites one that is still read.  The number of ring
slots and the order of the S issuer's waits are read from the kernels' sources.
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


def run(items, slots, waits, dual, seed):
    """`items`: key blocks of tile 0 and of tile 1 of each item (a pair of row
    tiles, or one).  One ring of K and V tiles in turn; `waits`: what the S issuer
    waits for, in its order; `dual`: a score buffer per tile."""
    rng = random.Random(seed)
    full, empty = [[Barrier() for _ in range(slots)] for _ in range(2)]
    s_full, s_free, p_full, pv_done = [[Barrier(), Barrier()] for _ in range(4)]
    q_full, q_empty = Barrier(), Barrier()
    copies, products = [], ([], [])  # products complete in the order of their issue
    tile, used = [None] * slots, [None] * slots

    def blocks():
        g = 0
        for n0, n1 in items:
            for j in range(max(n0, n1)):
                yield g, j, [t for t, n in enumerate((n0, n1)) if j < n], j == max(n0, n1) - 1
                g += 1

    def producer():
        def load(f):
            s, u = f % slots, f // slots
            if u:
                yield from wait(empty[s], u - 1)
            assert used[s] is None, ("a tile still in use is overwritten", f)
            full[s].expect()
            tile[s], used[s] = None, f

            def land():
                tile[s] = f
                full[s].land()

            copies.append(land)
            yield

        q = 0
        for g, j, _, _ in blocks():
            yield from load(2 * g)
            yield from load(2 * g + 1)
            if j == 0:
                if q:
                    yield from wait(q_empty, q - 1)
                q_full.expect()
                copies.append(q_full.land)
                q += 1

    def product(queue, f, barrier):
        def read():
            assert tile[f % slots] == f, ("a product reads another tile", tile[f % slots], f)

        queue.extend([read, barrier.arrive])

    def release(queue, f):
        def done():
            used[f % slots] = None
            empty[f % slots].arrive()

        queue.append(done)

    def s_issuer():
        q, uses, two_before = 0, [0, 0], False
        for g, j, tiles, last in blocks():
            f = 2 * g
            landed = False
            if j == 0:
                yield from wait(q_full, q)
                q += 1
            for t in tiles:
                b = t if dual else 0
                for what in waits:
                    if what == "free" and uses[b]:
                        yield from wait(s_free[b], uses[b] - 1)
                    elif (what == "here" or what == "here after two" and two_before) and not landed:
                        yield from wait(full[f % slots], f // slots)
                        landed = True
                product(products[0], f, s_full[t])
                uses[b] += 1
                yield
            two_before = len(tiles) == 2
            release(products[0], f)
            if last:
                products[0].append(q_empty.arrive)
            yield

    def pv_issuer():
        uses = [0, 0]
        for g, _, tiles, _ in blocks():
            f = 2 * g + 1
            yield from wait(full[f % slots], f // slots)
            for t in tiles:
                yield from wait(p_full[t], uses[t])
                product(products[1], f, pv_done[t])
                uses[t] += 1
                yield
            release(products[1], f)
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
    """Slots of the K/V ring at head dimension d, and the S issuer's waits in their
    order: for the score buffer ("free") and for K's tile ("here"; "here after
    two" where the block before had two row tiles)."""
    text = open(os.path.join(build.CSRC_DIR, source)).read()
    slots = re.search(r"kSlots = .*?\(?D == 128\)? \? (\d+) : (\d+)", text)
    issuer = text[text.index("- S issuer"):text.index("- P V issuer")]
    waits = []
    for line in re.findall(r".*wait_bounded_inl\(&bar->(?:s_free|kv_full)\[.*", issuer):
        waits.append("free" if "s_free" in line else "here after two" if "two_before" in line else "here")
    return int(slots.group(1 if d == 128 else 2)), waits


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
    slots, waits = ring(source, d)
    for seed in range(300):
        r = random.Random(seed)
        run(ITEMS[items](r.choice([1, 2, 4, 9, 30]), r), slots, waits, d == 64, seed)
