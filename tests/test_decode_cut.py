"""How the paged decode cuts a batch into equal runs, restated in Python after
fa_decode_kernel.cuh (the start of a run, its segments, the join's description):
with lengths that stay, every tile is taken once and every cut unit is joined from
exactly its parts; with lengths that change from read to read, every request, unit,
tile, column and slot stays in range and every loop ends."""
import random

import pytest

SEG_COST, SEG_COST_FOURS, MIN_RUN, FOURS_RUN, FOURS_SHORT = 8, 2, 8, 20, 32
THREADS = 128


def i32(x):
    return (x + 2 ** 31) % 2 ** 32 - 2 ** 31


def u32(x):
    return x % 2 ** 32


class Launch:
    def __init__(self, lens, HH, keys, width, shift, grid, token_major, read):
        self.B, self.HH, self.keys, self.width, self.shift = len(lens), HH, keys, width, shift
        self.grid, self.token_major, self.lens, self.read = grid, token_major, lens, read

    def len(self, b):
        assert 0 <= b < self.B
        return min(max(self.read(self.lens[b]), 0), self.width << self.shift)

    def tiles(self, n):
        return 1 if n <= self.keys else (n - 1) // self.keys + 1

    @staticmethod
    def start(total, workers, c):
        if total < 1 << 20:
            return u32(u32(total) * c) // workers
        return total * c // workers

    @staticmethod
    def worker_of(total, workers, tile):
        if total < 1 << 20:
            return i32(u32(u32(tile + 1) * workers - 1) // total)
        return i32(((tile + 1) * workers - 1) // total)


class Worker:
    """One block: its run, as (request, unit, t0, t1, tiles, key heads, the segment's slot or None) and its
    description for the join."""

    def __init__(self, p, worker):
        self.p, self.segments, self.meta = p, [], None
        per = (p.B + THREADS - 1) // THREADS
        spans = [(min(t * per, p.B), min(t * per + per, p.B)) for t in range(THREADS)]
        mine = [sum(p.tiles(p.len(b)) for b in range(*s)) for s in spans]
        tiles = sum(mine)
        fours = p.HH // 4
        self.units, self.cost, self.heads = p.HH, SEG_COST, 1
        if p.HH % 4 == 0 and (p.token_major or tiles <= p.B * FOURS_SHORT if p.B * fours >= p.grid else
                              p.token_major and tiles * fours >= p.grid * FOURS_RUN):
            self.units, self.cost, self.heads = fours, SEG_COST_FOURS, 4
        total = (tiles + p.B * self.cost) * self.units
        self.workers = workers = min(p.grid, (total + MIN_RUN - 1) // MIN_RUN)
        if worker >= workers:
            return
        begin, end = p.start(total, workers, worker), p.start(total, workers, worker + 1)
        found = []
        before = 0
        for (lo, hi), n in zip(spans, mine):
            at = (before + lo * self.cost) * self.units
            before += n
            if at <= begin < at + (n + (hi - lo) * self.cost) * self.units:
                b = lo
                while True:
                    assert b < hi
                    length = p.len(b)
                    n = (p.tiles(length) + self.cost) * self.units
                    if begin < at + n or b + 1 >= hi:
                        break
                    at += n
                    b += 1
                found.append((b, length, at))
        assert len(found) == 1                              # one thread claims the run
        self.b, self.len, at = found[0]
        self.nt = p.tiles(self.len)
        inside, unit = begin - at, self.nt + self.cost
        assert inside >= 0
        u = i32(u32(inside) // u32(unit)) if inside <= 0xffffffff else i32(inside // unit)
        self.u = min(u, self.units - 1)
        assert self.u >= 0
        x = i32(inside - self.u * unit)
        self.rem = end - begin
        self.take(x)
        if x > self.cost:
            u0 = begin - x
            first = max(0, min(p.worker_of(total, workers, u0 + self.cost), worker - 1))
            last = p.worker_of(total, workers, u0 + self.cost + self.nt - 1)
            self.meta = (self.b, self.u, 2 * first if p.start(total, workers, first) >= u0 else 2 * first + 1,
                         max(worker, min(last, workers - 1)), self.heads)
        first_seg = self.t0 < self.t1
        if not first_seg and not self.next():
            return
        while True:
            whole = self.t0 == 0 and self.t1 == self.nt
            slot = None if whole else 2 * worker + (0 if first_seg else 1)
            self.segments.append((self.b, self.u, self.t0, self.t1, self.nt, self.heads, slot))
            self.check()
            first_seg = False
            if not self.next():
                return

    def take(self, x):
        left = self.cost + self.nt - x
        n = i32(min(self.rem, left))
        self.t0, self.t1 = max(0, i32(x - self.cost)), max(0, i32(x + n - self.cost))
        self.rem -= n

    def next(self):
        while True:
            if self.rem <= 0:
                return False
            self.u += 1
            if self.u >= self.units:
                self.u, self.b = 0, self.b + 1
                if self.b >= self.p.B:
                    return False
                self.len = self.p.len(self.b)
                self.nt = self.p.tiles(self.len)
            self.take(0)
            if self.t0 < self.t1:
                return True

    def check(self):
        p = self.p
        assert 0 <= self.b < p.B and 0 <= self.u < self.units
        assert 0 <= self.t0 <= self.t1 <= self.nt
        last = self.t1 * p.keys - 16                        # the last 16-key group looked up, if it holds a key
        assert min(last, max(self.len - 1, 0)) >> p.shift < p.width
        head = self.u * self.heads + self.heads - 1
        assert head < p.HH


def check_join(p, c, meta):
    b, u, slot, last, heads = meta
    first = slot >> 1
    assert 0 <= b < p.B and 0 <= u * heads + heads - 1 < p.HH and 0 <= first < c <= last < p.grid
    for rows in (1, 8, 16):                                  # the elements of block c: all of them, and no other's
        everything, cuts = heads * rows * 32, last - first
        assert 0 <= everything * (c - first - 1) // cuts <= everything * (c - first) // cuts <= everything
    return [slot] + [2 * i for i in range(first + 1, last + 1)]


def batch(rng):
    B = rng.choice([1, 2, 3, 9, 64, 130, 300])
    top = rng.choice([1, 40, 700, 9000, 70000])
    shift = rng.choice([4, 6, 12])
    lens = [rng.choice([0, 1, rng.randint(0, top), top]) for _ in range(B)]
    width = max(1, -(-max(lens) >> shift)) + rng.choice([0, 0, 5, 4000])
    return dict(lens=lens, HH=rng.choice([1, 2, 4, 8, 12, 32]), keys=rng.choice([16, 32, 64]), width=width, shift=shift,
                grid=rng.choice([2, 7, 304, 304]), token_major=rng.random() < 0.6)


def test_every_tile_is_taken_once_and_joined():
    rng = random.Random(2)
    for _ in range(120):
        x = batch(rng)
        p = Launch(read=lambda n: n, **x)
        taken, joins = {}, {}
        for w in range(p.grid):
            k = Worker(p, w)
            for b, u, t0, t1, nt, heads, slot in k.segments:
                taken.setdefault((b, u), []).append((t0, t1, nt, slot))
            if k.meta:
                assert k.meta[3] < k.workers
                joins.setdefault(k.meta[:2], []).append((w, k.meta))
            units = k.units if k.segments else None
            assert units is None or all(s[5] * units == p.HH for s in k.segments)
        seen = {u for _, u in taken}
        assert set(taken) == {(b, u) for b in range(p.B) for u in range(max(seen) + 1)}
        for unit, parts in taken.items():
            at = 0
            for t0, t1, nt, _ in parts:                      # in the workers' order
                assert t0 == at and t1 > t0
                at = t1
            assert at == nt == p.tiles(p.len(unit[0]))
            slots = [s for _, _, _, s in parts]
            if len(parts) == 1:
                assert slots == [None] and unit not in joins
                continue
            for c, meta in joins[unit]:
                assert check_join(p, c, meta) == slots
            assert [c for c, _ in joins[unit]] == list(range((slots[0] >> 1) + 1, joins[unit][0][1][3] + 1))
        assert set(joins) <= set(taken)


@pytest.mark.parametrize("seed", range(4))
def test_lengths_that_change_stay_in_range(seed):
    rng = random.Random(100 + seed)
    for _ in range(25):
        x = batch(rng)
        wild = rng.choice([0.02, 0.3, 1.0])
        values = [0, 1, -5, 2 ** 31 - 1, -2 ** 31, 12345, 70000, 100, 17]

        def read(n):
            return rng.choice(values) if rng.random() < wild else n

        p = Launch(read=read, **x)
        for w in rng.sample(range(p.grid), min(p.grid, 12)):
            k = Worker(p, w)
            if k.meta:
                check_join(p, w, k.meta)


def test_the_longest_tables():
    """Lengths next to 2^31 and 2^27 tiles: 64-bit counts all through, and reads that
    fall from there to nothing."""
    rng = random.Random(9)
    for lens in ([2 ** 31 - 65537] * 3, [2 ** 31 - 65537] * 40, [1, 2 ** 31 - 65537, 0, 5]):
        for read in (lambda n: n, lambda n: rng.choice([n, n, 0, 1, 2 ** 31 - 1])):
            p = Launch(lens, 8, 16, (2 ** 31 - 65536) >> 16, 16, 304, True, read)
            for w in (0, 1, 2, 150, 302, 303):
                k = Worker(p, w)
                if k.meta:
                    check_join(p, w, k.meta)
