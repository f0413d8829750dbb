"""moe_attend8's warps and barriers as a model on the CPU: coroutines on a random
scheduler, mbarriers by phase and parity, copies and products that end after random
times. Every tile must find its own keys, values, pages and scales, no barrier may be
arrived at more often than a phase counts, and all parts must end. The stages of
the rings are those of csrc/attend8.cu."""
import heapq
import os
import random
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "moe_expert_layer_warp_gb300", "csrc", "attend8.cu")
SLOTS, PARTS = 16, 8


def stages():
    """(keys' stages, values') of every size that the source has."""
    text = open(SOURCE).read()
    found = [re.search(r"%s = kDim == 64 \? (\d+) : ([^;]*);" % name, text)
             for name in ("kKeyStages", "kValueStages")]
    wide = [[int(v) for v in re.findall(r"\d+", m.group(2).replace("kNum == 2", ""))]
            for m in found]
    sizes = {(int(found[0].group(1)), int(found[1].group(1)))}
    for i in range(max(map(len, wide))):
        sizes.add(tuple(w[min(i, len(w) - 1)] for w in wide))
    return sorted(sizes)


class Barrier:
    def __init__(self, count):
        self.count = self.pending = count
        self.bytes = self.phase = 0

    def arrive(self, n=1, expect=0):
        assert self.pending >= n, "more arrivals than a phase counts"
        self.pending -= n
        self.bytes += expect
        self.turn()

    def landed(self, n):
        self.bytes -= n
        self.turn()

    def turn(self):
        if self.pending == 0 and self.bytes == 0:
            self.phase, self.pending = self.phase + 1, self.count

    def test(self, parity):
        return self.phase & 1 != parity


class Model:
    """`parts`: (tiles, log2 of the streams) of the parts of a CTA's range. keys,
    values: stages of the two rings; values None: one ring for both."""

    def __init__(self, parts, keys, values, seed):
        self.rng = random.Random(seed)
        self.parts, self.keys, self.values = parts, keys, values
        self.now, self.events, self.order = 0, [], 0
        n = keys + (values or 0)
        self.full, self.empty = ([Barrier(1) for _ in range(n)] for _ in range(2))
        self.part_full = [Barrier(1) for _ in range(PARTS)]
        self.part_empty = [Barrier(19) for _ in range(PARTS)]
        self.raw_full, self.raw_empty, self.q_full = Barrier(32), Barrier(16), Barrier(16)
        self.pages, self.scales, self.done = ([Barrier(1) for _ in range(SLOTS)] for _ in range(3))
        self.s_full, self.p_done = ([Barrier(1) for _ in range(4)] for _ in range(2))
        self.s_empty, self.p_full = ([Barrier(16) for _ in range(4)] for _ in range(2))
        self.part, self.slot, self.stage = [None] * PARTS, [None] * SLOTS, [None] * n
        self.queries, self.converted, self.pipe, self.syncs = None, 0, 0, {}
        self.copy = self.rng.choice([(1, 3), (5, 60), (50, 300), (1, 300)])
        self.product = self.rng.choice([(1, 3), (1, 20), (10, 10)])

    # -- time
    def later(self, ticks, what):
        self.order += 1
        heapq.heappush(self.events, (self.now + ticks, self.order, what))

    def issue(self, barriers):
        """A product, done in order behind those before it."""
        self.pipe = max(self.pipe, self.now) + self.rng.randint(*self.product)
        for b in barriers:
            self.later(self.pipe - self.now, b.arrive)

    def some(self, most):
        return self.rng.randint(1, most)

    def wait(self, barrier, parity):
        while not barrier.test(parity):
            yield None

    def sync(self, name, n):
        s = self.syncs.setdefault(name, [0, 0])
        turn = s[1]
        s[0] += 1
        if s[0] == n:
            s[0], s[1] = 0, turn + 1
        while s[1] == turn:
            yield None

    # -- places
    def place(self, kind, tile, part_place, j, streams, n):
        """(stage, parity of its filling) of a part's tile j."""
        if self.values is not None:
            count, first = (self.keys, 0) if kind == "K" else (self.values, self.keys)
            return first + tile % count, tile // count & 1
        if kind == "K":
            at = part_place + (j if j < streams else 2 * j - streams)
        else:
            at = part_place + (2 * j + streams + 1 if j + streams < n else n + j)
        return at % self.keys, at // self.keys & 1

    @staticmethod
    def add(counts, n, shift):
        return [c + (((n - 1 - s) >> shift) + 1 if s >> shift == 0 and n > s else 0)
                for s, c in enumerate(counts)]

    def walk(self):
        """Every part as (number, tiles, log2 streams, first tile, first place)."""
        tile = 0
        for no, (n, shift) in enumerate(self.parts):
            yield no, n, shift, tile, 2 * tile
            tile += n

    def take(self, no):
        yield from self.wait(self.part_full[no % PARTS], no // PARTS & 1)
        assert self.part[no % PARTS] == (self.parts[no] if no < len(self.parts) else None)

    # -- roles
    def loader(self):
        for no, n, shift, tile, first in self.walk():
            yield from self.take(no)
            streams = 1 << shift
            for j in range(-streams, n):
                want = [("K", j + streams)] if j + streams < n else []
                want += [("V", j)] if j >= 0 else []
                at = {}
                for kind, i in want:
                    if kind == "K":
                        yield from self.wait(self.pages[(tile + i) % SLOTS],
                                             (tile + i) // SLOTS & 1)
                    at[kind], parity = self.place(kind, tile + i, first, i, streams, n)
                    yield from self.wait(self.empty[at[kind]], parity ^ 1)
                for kind, i in want:
                    assert self.slot[(tile + i) % SLOTS] == tile + i
                    b = self.full[at[kind]]
                    self.stage[at[kind]] = (kind, tile + i)
                    b.arrive(1, 2)
                    for _ in range(2):
                        self.later(self.rng.randint(*self.copy), lambda b=b: b.landed(1))
                yield 1
            self.part_empty[no % PARTS].arrive()

    def products(self, scores):
        counts = [0] * 4
        for no, n, shift, tile, first in self.walk():
            yield from self.take(no)
            streams = 1 << shift
            if scores:
                for s in range(4):
                    yield from self.wait(self.s_empty[s], counts[s] & 1 ^ 1)
                yield from self.wait(self.q_full, no & 1)
            for j in range(n):
                s, kind = j % streams, "K" if scores else "V"
                k = counts[s] + (j >> shift)
                at, parity = self.place(kind, tile + j, first, j, streams, n)
                if scores:
                    yield from self.wait(self.full[at], parity)
                    yield from self.wait(self.scales[(tile + j) % SLOTS], (tile + j) // SLOTS & 1)
                    yield from self.wait(self.s_empty[s], k & 1 ^ 1)
                    assert self.queries == no
                    ends = [self.s_full[s], self.empty[at]]
                else:
                    yield from self.wait(self.p_full[s], k & 1)
                    yield from self.wait(self.full[at], parity)
                    ends = [self.p_done[s], self.empty[at], self.done[(tile + j) % SLOTS]]
                assert self.stage[at] == (kind, tile + j) and self.full[at].bytes == 0
                self.issue(ends)
                yield 1
            counts = self.add(counts, n, shift)
            self.part_empty[no % PARTS].arrive()

    def ahead(self):
        total = sum(n for n, _ in self.parts)
        ends = [sum(n for n, _ in self.parts[:i + 1]) for i in range(len(self.parts))]
        published = queries = tiles = asked = group = 0
        while published <= len(self.parts) or queries <= len(self.parts) or tiles < total:
            here = next((i for i, e in enumerate(ends) if asked < e), len(self.parts))
            if published <= len(self.parts) and published < min(queries, here) + PARTS - 1 and (
                    self.part_empty[published % PARTS].test(published // PARTS & 1 ^ 1)):
                self.part[published % PARTS] = (self.parts + [None])[published]
                self.part_full[published % PARTS].arrive()
                published += 1
            known = ends[min(published, len(self.parts)) - 1] if published else 0
            if not group:
                group = min(4, known - asked)
                asked += group
            if queries < published and self.raw_empty.test(queries & 1 ^ 1):
                for _ in range(32):
                    self.later(self.some(20), self.raw_full.arrive)
                queries += 1
            last = tiles + group - 1
            if group and self.done[last % SLOTS].test(last // SLOTS & 1 ^ 1):
                mine = range(tiles, tiles + group)
                for i in mine:
                    self.slot[i % SLOTS] = i
                    self.pages[i % SLOTS].arrive()
                tiles += group
                group = min(4, known - asked)
                asked += group
                yield self.some(8)
                for i in mine:
                    self.scales[i % SLOTS].arrive()
            yield 1

    def softmax(self, warp):
        group, counts, part = warp // 4, [0] * 4, None
        for then in list(self.walk()) + [None]:
            no = then[0] if then else len(self.parts)
            yield from self.take(no)
            yield from self.wait(self.raw_full, no & 1)
            if then:
                yield self.some(5)
                self.converted += 1
                if self.converted % 16 == 0:
                    self.queries = no
                self.raw_empty.arrive()
                self.q_full.arrive()
            for s in range(4):
                yield from self.wait(self.p_done[s], counts[s] & 1 ^ 1)
            yield from self.sync("all", 16)
            if part is not None:
                assert [b.phase for b in self.p_done] == counts   # the results are there
                for _ in range(2):
                    yield self.some(10)
                    yield from self.sync("all", 16)
                self.part_empty[part % PARTS].arrive()
            if not then:
                return
            part, n, shift, tile, first = then
            streams, s = 1 << shift, group >> (2 - shift)
            yield from self.sync("all", 16)
            for k, j in enumerate(range(s, n, streams), counts[s]):
                yield from self.wait(self.s_full[s], k & 1)
                assert self.slot[(tile + j) % SLOTS] == tile + j and self.s_full[s].phase == k + 1
                yield self.some(4)
                self.s_empty[s].arrive(streams)
                yield from self.sync(group, 4)
                yield from self.wait(self.p_done[s], k & 1 ^ 1)
                if j == n - 1 or self.rng.random() < 0.1:         # values to be cleaned
                    at, parity = self.place("V", tile + j, first, j, streams, n)
                    yield from self.wait(self.full[at], parity)
                    assert self.stage[at] == ("V", tile + j) and self.full[at].bytes == 0
                yield self.some(4)
                self.p_full[s].arrive(streams)
            counts = self.add(counts, n, shift)
            for i in range(4):
                yield from self.wait(self.s_full[i], counts[i] & 1 ^ 1)

    def run(self):
        roles = [self.loader(), self.products(True), self.products(False), self.ahead()]
        roles += [self.softmax(w) for w in range(16)]
        wake, idle = [0] * len(roles), 0
        while any(roles):
            while self.events and self.events[0][0] <= self.now:
                heapq.heappop(self.events)[2]()
            moved = bool(self.events)
            for i in self.rng.sample(range(len(roles)), len(roles)):
                if roles[i] is None or wake[i] > self.now:
                    moved |= roles[i] is not None
                    continue
                try:
                    ticks = next(roles[i])
                except StopIteration:
                    roles[i], ticks = None, 1
                wake[i] = self.now + (ticks or 0)
                moved |= ticks is not None and i != 3             # (the warp ahead polls)
            self.now += 1
            idle = 0 if moved else idle + 1
            assert idle < 50, "no role goes on"


def ranges(seed):
    rng = random.Random(seed)
    return [(rng.choice([1, 2, 3, 4, 5, 7, rng.randint(1, 44)]),
             2 if seed % 4 < 2 else rng.choice([2, 2, 1, 0])) for _ in range(rng.randint(2, 12))]


@pytest.mark.parametrize("keys, values", stages())
def test_every_tile_finds_its_own(keys, values):
    for seed in range(100):
        Model(ranges(seed), keys, values, seed).run()


def test_the_model_sees_a_ring_for_both():
    """One ring of 9 stages: the warp with the scores takes a stage that still waits
    for values of the turn before."""
    with pytest.raises(AssertionError):
        for seed in range(100):
            Model(ranges(seed), 9, None, seed).run()


def test_the_sources_stages_are_found():
    assert len(stages()) >= 2 and all(k >= 2 and v >= 4 for k, v in stages())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_many_items_a_cta(dtype):
    """Eight and more items of few rows for every CTA, calls one after the other
    without a pause: the same bits every time, and within their bound."""
    import torch
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from moe_expert_layer_warp_gb300 import api, build
    from tests.test_kv8_ops import Attend
    build.build()
    a = Attend([1 + i % 2 for i in range(150)], [100 + 37 * i for i in range(150)], 32, 8, 128,
               getattr(torch, dtype), 64, block=64)
    r, args = a.runner(), a.args()
    first = r.attend(*args).clone()
    outs = [torch.full_like(first, 7.0) for _ in range(40)]
    for out in outs:
        r.attend(*args, out=out)
    assert api.moe_last_device_error() == api.MOE_OK
    a.check(first)
    for out in outs:
        assert torch.equal(out.view(torch.int16), first.view(torch.int16))
