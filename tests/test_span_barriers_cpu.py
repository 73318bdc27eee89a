"""The span kernels' barriers, as models on the CPU (see test_barrier_model_cpu): row tiles
that take different blocks of an item, blocks that no tile takes, rows of V that are
zeroed in between, and the kernel for few rows.  The ring's slots are read from the
kernels' sources."""

import os
import random
import re

import pytest

from exact_tiled_attention_08_gb300 import build
from test_barrier_model_cpu import Barrier, ring, wait


class Counted(Barrier):
    """A barrier that takes several arrivals a phase."""

    def __init__(self, count):
        self.count = count
        self.pending, self.copies, self.phase = count, 0, 0

    def step(self):
        if self.pending == 0 and self.copies == 0:
            self.phase += 1
            self.pending = self.count


def interleave(roles, copies, products, rng, speeds):
    """Runs the roles in random turns; copies land in any order, products complete in the order of their issue."""
    speed = {name: rng.choice([1, 1, 5, 20]) for name in speeds}
    in_order, steps = rng.random(), 0
    while roles or copies or any(products):
        steps += 1
        assert steps < 400000, "no role can go on"
        names = [*roles, *(["copies"] if copies else []), *(i for i, x in enumerate(products) if x)]
        name = rng.choices(names, [speed[n] for n in names])[0]
        if name == "copies":
            copies.pop(0 if rng.random() < in_order else rng.randrange(len(copies)))()
        elif isinstance(name, int):
            products[name].pop(0)()
        else:
            try:
                next(roles[name])
            except StopIteration:
                del roles[name]


class Ring:
    """K and V tiles with slots of their own."""

    def __init__(self, slots, copies):
        self.slots, self.copies = slots, copies
        self.full, self.empty = [[Barrier() for _ in range(sum(slots))] for _ in range(2)]
        self.tile, self.used = [None] * sum(slots), [None] * sum(slots)

    def place(self, kv, g):
        return kv * self.slots[0] + g % self.slots[kv], g // self.slots[kv]

    def load(self, kv, g):
        s, u = self.place(kv, g)
        if u:
            yield from wait(self.empty[s], u - 1)
        assert self.used[s] is None, ("a tile still in use is overwritten", kv, g)
        self.full[s].expect()
        self.tile[s], self.used[s] = None, (kv, g)

        def land():
            self.tile[s] = kv, g
            self.full[s].land()

        self.copies.append(land)
        yield

    def landed(self, kv, g):
        s, u = self.place(kv, g)
        yield from wait(self.full[s], u)

    def read(self, kv, g):
        assert self.tile[self.place(kv, g)[0]] == (kv, g), ("another tile is read", kv, g)

    def release(self, kv, g):
        self.used[self.place(kv, g)[0]] = None
        self.empty[self.place(kv, g)[0]].arrive()


def run_pairs(items, slots, dual, paged, seed):
    """`items`: of each the blocks, each tile's range of them (None: no such tile), and which are dirty.
    `paged`: K and V are loaded by two roles, else the second one only zeroes rows of V."""
    rng = random.Random(seed)
    copies, products = [], [[], []]
    tiles = Ring(slots, copies)
    s_full, s_free, p_full, pv_done = [[Barrier(), Barrier()] for _ in range(4)]
    q_full, q_empty, v_ask, v_clean = [Barrier() for _ in range(4)]
    segments = 4
    seg_full, seg_empty = [Barrier() for _ in range(segments)], [Counted(11) for _ in range(segments)]
    cleaned = set()

    def segment(n):
        yield from wait(seg_full[n % segments], n // segments)

    def active(item, j):
        return [t for t, r in enumerate(item["tiles"]) if r and r[0] <= j < r[1]]

    def producer():
        g = 0
        for n, item in enumerate([*items, None]):
            if n >= segments:
                yield from wait(seg_empty[n % segments], n // segments - 1)
            seg_full[n % segments].arrive()
            yield
            if item is None:
                return
            for j in range(item["blocks"]):
                yield from tiles.load(0, g)
                if not paged:
                    yield from tiles.load(1, g)
                if j == 0:
                    if n:
                        yield from wait(q_empty, n - 1)
                    q_full.expect()
                    copies.append(q_full.land)
                g += 1

    def values():
        g, asked, unseen, of = 0, 0, None, 0

        def clean():
            yield from wait(v_ask, asked)
            tiles.read(1, unseen)
            cleaned.add(unseen)
            yield
            v_clean.arrive()

        for n, item in enumerate(items):
            if unseen is not None and (not paged or n - of > 1):
                yield from clean()
                asked, unseen = asked + 1, None
            yield from segment(n)
            seg_empty[n % segments].arrive()
            for j in range(item["blocks"]):
                dirty = j in item["dirty"]
                if unseen is not None and (dirty or not paged or g - unseen >= slots[1]):
                    yield from clean()
                    asked, unseen = asked + 1, None
                if paged:
                    yield from tiles.load(1, g)
                if dirty:
                    unseen, of = g, n
                g += 1
        if unseen is not None:
            yield from clean()

    def s_issuer():
        g, uses = 0, [0, 0]
        for n, item in enumerate(items):
            yield from segment(n)
            seg_empty[n % segments].arrive()
            yield from wait(q_full, n)
            for j in range(item["blocks"]):
                yield from tiles.landed(0, g)
                for t in active(item, j):
                    b = t if dual else 0
                    if uses[b]:
                        yield from wait(s_free[b], uses[b] - 1)
                    products[0].extend([lambda g=g: tiles.read(0, g), s_full[t].arrive])
                    uses[b] += 1
                    yield
                products[0].append(lambda g=g: tiles.release(0, g))
                g += 1
                yield
            products[0].append(q_empty.arrive)

    def pv_issuer():
        g, uses, cleans = 0, [0, 0], 0

        def read(g, dirty):
            tiles.read(1, g)
            assert not dirty or g in cleaned, ("a product reads rows that are to be zeroed", g)

        for n, item in enumerate(items):
            yield from segment(n)
            seg_empty[n % segments].arrive()
            for j in range(item["blocks"]):
                yield from tiles.landed(1, g)
                dirty = j in item["dirty"]
                clean = not dirty
                if dirty:
                    v_ask.arrive()
                for t in active(item, j):
                    yield from wait(p_full[t], uses[t])
                    if not clean:
                        yield from wait(v_clean, cleans)
                        clean = True
                    products[1].extend([lambda g=g, dirty=dirty: read(g, dirty), pv_done[t].arrive])
                    uses[t] += 1
                    yield
                if not clean:
                    yield from wait(v_clean, cleans)
                cleans += dirty
                products[1].append(lambda g=g: tiles.release(1, g))
                g += 1
                yield

    def softmax(t):
        uses = 0
        for n, item in enumerate(items):
            yield from segment(n)
            r = item["tiles"][t]
            for j in range(*r) if r else ():
                yield from wait(s_full[t], uses)
                s_free[t if dual else 0].arrive()
                yield
                if j > r[0]:
                    yield from wait(pv_done[t], uses - 1)
                p_full[t].arrive()
                uses += 1
                yield
            if r:
                yield from wait(pv_done[t], uses - 1)
            for _ in range(4):  # (its warps)
                seg_empty[n % segments].arrive()

    roles = {f.__name__: f() for f in (producer, values, s_issuer, pv_issuer)}
    roles.update({"softmax 0": softmax(0), "softmax 1": softmax(1)})
    interleave(roles, copies, products, rng, [*roles, "copies", 0, 1])


def random_items(r):
    """Items whose tiles take the same blocks, shifted ones, ones with a gap between them, or one tile alone."""
    items = []
    for _ in range(r.choice([1, 2, 6, 9])):
        n = r.choice([1, 2, 3, 4, 9])
        a, b = sorted((r.randint(0, n), r.randint(0, n)))
        tiles = r.choice([[(0, n), (0, n)], [(0, n), None], [(0, max(1, n - 1)), (min(1, n - 1), n)],
                          [(0, max(1, a)), (min(b, n - 1), n)]])
        items.append({"blocks": n, "tiles": tiles, "dirty": {j for j in (0, n - 1) if r.random() < 0.4}})
    return items


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_no_wait_passes_early_in_pairs(d, paged):
    for seed in range(150):
        r = random.Random(seed)
        run_pairs(random_items(r), ring("fa_cross_fwd.cuh", d), d == 64, paged, seed)


def few_slots(d):
    text = open(os.path.join(build.CSRC_DIR, "fa_span_few.cuh")).read()
    k = re.search(r"kKSlots = D == 128 \? (\d+) : (\d+), kVSlots = kKSlots", text)
    return (int(k[1 if d == 128 else 2]),) * 2


def run_few(items, slots, seed):
    """`items`: the blocks of each segment; a block in random places moves the reference."""
    rng = random.Random(seed)
    copies, products = [], [[]]
    tiles = Ring(slots, copies)
    s_full, s_free, p_full, pv_done, q_full, q_empty = [[Barrier(), Barrier()] for _ in range(6)]
    moves = random.Random(seed + 1)

    def producer():
        g = 0
        for n, blocks in enumerate(items):
            for j in range(blocks):
                yield from tiles.load(0, g)
                if j == 0:
                    if n >= 2:
                        yield from wait(q_empty[n & 1], (n >> 1) - 1)
                    q_full[n & 1].expect()
                    copies.append(q_full[n & 1].land)
                g += 1

    def values():
        for g in range(sum(items)):
            yield from tiles.load(1, g)

    def issuer():
        g = 0
        for n, blocks in enumerate(items):
            yield from wait(q_full[n & 1], n >> 1)
            for i in range(blocks + 1):
                if i < blocks:
                    k = g + i
                    yield from tiles.landed(0, k)
                    if k >= 2:
                        yield from wait(s_free[k & 1], (k >> 1) - 1)
                    products[0].extend([lambda k=k: tiles.read(0, k), s_full[k & 1].arrive, lambda k=k: tiles.release(0, k)])
                    if i == blocks - 1:
                        products[0].append(q_empty[n & 1].arrive)
                    yield
                if i:
                    k = g + i - 1
                    yield from tiles.landed(1, k)
                    yield from wait(p_full[k & 1], k >> 1)
                    products[0].extend([lambda k=k: tiles.read(1, k), pv_done[k & 1].arrive, lambda k=k: tiles.release(1, k)])
                    yield
            g += blocks

    def softmax():
        g = 0
        for blocks in items:
            for j in range(blocks):
                yield from wait(s_full[g & 1], g >> 1)
                s_free[g & 1].arrive()
                yield
                if j and moves.random() < 0.3:
                    yield from wait(pv_done[(g - 1) & 1], (g - 1) >> 1)
                if g >= 2:
                    yield from wait(pv_done[g & 1], (g >> 1) - 1)
                if moves.random() < 0.2:  # rows of V are zeroed
                    yield from tiles.landed(1, g)
                    tiles.read(1, g)
                p_full[g & 1].arrive()
                g += 1
                yield
            yield from wait(pv_done[(g - 1) & 1], (g - 1) >> 1)

    roles = {f.__name__: f() for f in (producer, values, issuer, softmax)}
    interleave(roles, copies, products, rng, [*roles, "copies", 0])


@pytest.mark.parametrize("d", [64, 128])
def test_no_wait_passes_early_with_few_rows(d):
    for seed in range(150):
        r = random.Random(seed)
        run_few([r.choice([1, 1, 2, 3, 7, 30]) for _ in range(r.choice([1, 2, 5, 9]))], few_slots(d), seed)
