"""The barriers of the attention behind shared prefixes, simulated with random delays.

A model of the attend kernel's warps (loads, conversions, queries, tensor-core issue, rows) and of
what arrives asynchronously (tiles, finished products).  Every wait checks that it is not passed by
the parity of the phase two before (or missed by two), every arrival that its barrier still expects
one, every reader that it finds what it wants, and the end that nothing is left in flight.  A model
with one `full` barrier an entry for both slots, as the kernel once had, fails."""
import heapq
import random

import pytest

UNITS, STEPS_AHEAD = 4, 8


class Fault(Exception):
    pass


class Bar:
    """An mbarrier: `count` arrivals complete a phase."""

    def __init__(self, name, count):
        self.name, self.count, self.left, self.phase = name, count, count, 0

    def arrive(self):
        if self.left <= 0:
            raise Fault("arrival too many: " + self.name)
        self.left -= 1
        if self.left == 0:
            self.phase, self.left = self.phase + 1, self.count

    def passed(self, n):
        """A test of the parity of phase n."""
        ok = self.phase & 1 != n & 1
        if ok and self.phase <= n:
            raise Fault("passed early: " + self.name)
        if not ok and self.phase > n + 1:
            raise Fault("missed: " + self.name)
        return ok


def wait(bar, n):
    while not bar.passed(n):
        yield None


class Kernel:
    """One CTA: runs of an A share (both slots), and of the slots' B shares as (blocks, rows)."""

    def __init__(self, rng, runs_a, rows_a, runs_b, f8, shared_full=False):
        self.rng, self.f8, self.shared = rng, f8, shared_full
        self.entries, self.codes = (4, 2) if f8 else (5, 0)
        self.runs_a, self.rows_a, self.runs_b = runs_a, rows_a, runs_b
        self.na, self.nb = sum(runs_a), [sum(n for n, _ in r) for r in runs_b]

        def bars(name, n, count):
            return [Bar("%s %d" % (name, i), count) for i in range(n)]

        self.full = [bars("full%d" % s, self.entries, 4 if f8 else 1) for s in (0, 1)]
        self.empty = bars("empty", self.entries, 2)
        self.code_full, self.code_empty = bars("code_full", 2, 1), bars("code_empty", 2, 4)
        self.s_full, self.p_full = bars("s_full", 2, 1), bars("p_full", 2, 4)
        self.o_full = bars("o_full", 2, 1)
        self.q_full = [bars("q_full%d" % s, UNITS, 1) for s in (0, 1)]
        self.q_done = [bars("q_done%d" % s, 2, 1) for s in (0, 1)]
        self.a_done = Bar("a_done", 1)
        self.ring, self.code = [None] * self.entries, [None, None]
        self.unit, self.half = [[None] * UNITS, [None] * UNITS], [[None, None], [None, None]]
        self.step = {}
        self.now, self.end, self.events, self.in_flight, self.tensor = 0, False, [], 0, 0

    def later(self, dt, f):
        self.in_flight += 1

        def event():
            self.in_flight -= 1
            f()

        heapq.heappush(self.events, (self.now + dt, self.rng.random(), event))

    def full_of(self, slot, x):
        return self.full[0 if self.shared else slot][x]

    def entry_b(self, s, k):
        return 2 * (self.na + k + min(k if s == 0 else k + 1, self.nb[1 - s]))

    def order(self):
        """Steps in the order of their loads: (slot whose barriers say so, key)."""
        for k in range(self.na):
            yield 0, ("A", k)
        left, at = list(self.nb), 0 if self.nb[0] else 1
        while left[0] or left[1]:
            k = self.nb[at] - left[at]
            assert self.entry_b(at, k) == 2 * (sum(self.nb) - sum(left) + self.na)
            yield at, (at, k)
            left[at] -= 1
            if left[1 - at]:
                at = 1 - at

    def loads(self):
        e, last = 0, {}
        uses = [[0] * self.entries, [0] * self.entries]
        for slot, key in self.order():
            w = 0 if self.shared else slot
            old = self.step.get(e // 2 % STEPS_AHEAD)
            if old and old["readers"] > 0:
                raise Fault("step overwritten")
            self.step[e // 2 % STEPS_AHEAD] = dict(key=key, slot=slot, readers=0,
                                                   v=uses[w][(e + 1) % self.entries])
            for side in "KV":
                x = e % self.entries
                bars, empty, n = (self.full[w], self.empty, self.entries)
                place, tiles = x, self.ring
                if self.f8:
                    place, tiles, n = e % 2, self.code, 2
                    bars, empty = self.code_full, self.code_empty
                if e >= n:
                    yield from wait(empty[place], e // n - 1)
                if tiles[place] is not None:
                    raise Fault("tile overwritten")

                def land(place=place, tile=(key, side), tiles=tiles, bar=bars[place]):
                    tiles[place] = tile
                    bar.arrive()

                last[place] = (bars[place], e // n if self.f8 else uses[w][x])
                uses[w][x] += 1
                yield self.rng.choice([0, 0, 1])
                self.later(self.rng.choice([5, 20, 200, 2000]), land)
                e += 1
        for place in range(self.entries if not self.f8 else 2):
            if place in last:
                yield from wait(*last[place])
        if not self.f8:
            for i in range(max(0, e - self.entries), e):
                yield from wait(self.empty[i % self.entries], i // self.entries)

    def converts(self):
        tiles = 2 * (self.na + sum(self.nb))
        for e in range(tiles):
            c, x = e % 2, e % self.entries
            yield from wait(self.code_full[c], e // 2)
            step, tile = self.step[e // 2 % STEPS_AHEAD], self.code[c]
            if tile[0] != step["key"]:
                raise Fault("step of another tile")
            yield self.rng.choice([1, 30])
            if self.code_empty[c].left == 1:
                self.code[c] = None
            self.code_empty[c].arrive()
            if e >= self.entries:
                yield from wait(self.empty[x], e // self.entries - 1)
            if self.ring[x] not in (None, tile):
                raise Fault("entry overwritten")
            self.ring[x] = tile
            yield self.rng.choice([1, 30, 100])
            self.full_of(step["slot"], x).arrive()
        for e in range(max(0, tiles - self.entries), tiles):
            yield from wait(self.empty[e % self.entries], e // self.entries)

    def queries(self):
        count, before = [0, 0], [0, 0]
        for part in (0, 1):
            runs = [[(n, self.rows_a[s]) for n in self.runs_a] if part == 0 else self.runs_b[s]
                    for s in (0, 1)]
            at = [0, 0]
            while at[0] < len(runs[0]) or at[1] < len(runs[1]):
                for s in (0, 1):
                    if at[s] == len(runs[s]):
                        continue
                    (run, rows), n = runs[s][at[s]], count[s]
                    room = n < 2 or self.q_done[s][n & 1].passed((n >> 1) - 1)
                    if n >= 1 and (rows > 64 or before[s] > 64):
                        room = room and self.q_done[s][~n & 1].passed((n - 1) >> 1)
                    if not room:
                        continue
                    row0 = (n + s & 1) * 64 if rows <= 64 else 0
                    old = self.unit[s][n % UNITS]
                    if old and old["readers"] < 5:  # four row warps and the issuing one
                        raise Fault("run overwritten")
                    halves = [row0 // 64] if rows <= 64 else [0, 1]
                    if any(self.half[s][h] and not self.half[s][h]["done"] for h in halves):
                        raise Fault("queries overwritten")
                    unit = dict(n=n, run=run, rows=rows, row0=row0, readers=0, done=False)
                    self.unit[s][n % UNITS] = unit
                    for h in halves:
                        self.half[s][h] = unit
                    yield self.rng.choice([3, 30, 300])
                    self.q_full[s][n % UNITS].arrive()
                    count[s], before[s], at[s] = n + 1, rows, at[s] + 1
                yield None
        for s in (0, 1):
            for n in range(max(0, count[s] - 2), count[s]):
                yield from wait(self.q_done[s][n & 1], n >> 1)

    def product(self, dt, arrivals):
        self.tensor = max(self.tensor, self.now) + dt
        for f in arrivals:
            self.later(self.tensor - self.now + self.rng.choice([1, 1, 5, 40]), f)

    def free(self, x):
        if self.empty[x].left == 1:
            self.ring[x] = None
        self.empty[x].arrive()

    def issues(self, warp):
        seen = [0] * self.entries
        state = [dict(n=0, left=0, unit=None) for _ in (0, 1)]

        def tile(s, e, both, side, k):
            x = e % self.entries
            if self.shared:
                yield from wait(self.full[0][x], e // self.entries)
            else:
                yield from wait(self.full[warp][x], seen[x])
            if self.ring[x] != (("A", k) if both else (s, k - self.na), side):
                raise Fault("another tile")
            if not both or s == 1:
                seen[x] += 1

        def scores(s, k, e, both):
            st, x = state[s], e % self.entries
            if st["left"] == 0:
                yield from wait(self.q_full[s][st["n"] % UNITS], st["n"] // UNITS)
                u = st["unit"] = self.unit[s][st["n"] % UNITS]
                if u["n"] != st["n"]:
                    raise Fault("another run")
                u["readers"] += 1
                st["left"], st["n"] = u["run"], st["n"] + 1
            yield from tile(s, e, both, "K", k)
            if k > 0:
                yield from wait(self.o_full[s], k - 1)
            st["left"] -= 1
            yield self.rng.choice([0, 1, 50])
            arrivals = [self.s_full[s].arrive]
            if st["left"] == 0:
                def done(unit=st["unit"], bar=self.q_done[s][~st["n"] & 1]):
                    unit["done"] = True
                    bar.arrive()
                arrivals.append(done)
            self.product(8, arrivals + [lambda: self.free(x)] * (1 if both else 2))

        def values(s, k, e, both):
            x = e % self.entries
            yield from tile(s, e, both, "V", k)
            yield from wait(self.p_full[s], k)
            yield self.rng.choice([0, 1, 50])
            self.product(16, [self.o_full[s].arrive] + [lambda: self.free(x)] * (1 if both else 2))

        if warp == 0 and self.na:
            for s in (0, 1):
                yield from scores(s, 0, 0, True)
            for k in range(self.na):
                for s in (0, 1):
                    yield from values(s, k, 2 * k + 1, True)
                    if k + 1 < self.na:
                        yield from scores(s, k + 1, 2 * k + 2, True)
            self.a_done.arrive()
        elif warp == 1:
            state[1]["n"] = len(self.runs_a)
            if self.na:
                yield from wait(self.a_done, 0)
        for k in range(self.nb[warp]):
            e = self.entry_b(warp, k)
            yield from scores(warp, self.na + k, e, False)
            yield from values(warp, self.na + k, e + 1, False)

    def rows(self, s, quarter):
        k = n = 0
        while k < self.na + self.nb[s]:
            yield from wait(self.q_full[s][n % UNITS], n // UNITS)
            u = self.unit[s][n % UNITS]
            if u["n"] != n:
                raise Fault("another run")
            yield self.rng.choice([0, 1, 100])
            u["readers"] += 1
            first, last = u["row0"] // 32, (u["row0"] + u["rows"] + 31) // 32
            for k in range(k, k + u["run"]):
                yield from wait(self.s_full[s], k)
                if not first <= quarter < last:
                    yield self.rng.choice([0, 1, 100])
                    self.p_full[s].arrive()
                    continue
                b = k >= self.na
                e = self.entry_b(s, k - self.na) if b else 2 * k
                step = self.step[e // 2 % STEPS_AHEAD]
                if step["key"] != ((s, k - self.na) if b else ("A", k)):
                    raise Fault("another step")
                step["readers"] += 1
                if not self.f8 and self.rng.random() < 0.5:  # a last block: V behind its end
                    yield from wait(self.full_of(s if b else 0, (e + 1) % self.entries), step["v"])
                yield self.rng.choice([5, 20, 400])
                step["readers"] -= 1
                self.p_full[s].arrive()
                yield from wait(self.o_full[s], k)
                yield self.rng.choice([1, 3, 200])
            k, n = k + 1, n + 1
            yield self.rng.choice([1, 10, 500])

    def run(self):
        warps = [self.loads(), self.queries(), self.issues(0), self.issues(1)]
        warps += [self.rows(s, q) for s in (0, 1) for q in range(4)]
        warps += [self.converts() for _ in range(4 if self.f8 else 0)]
        ready, alive, idle = [(0, i) for i in range(len(warps))], len(warps), 0
        while alive:
            if self.events and self.events[0][0] <= ready[0][0]:
                self.now, _, event = heapq.heappop(self.events)
                event()
                idle = 0
                continue
            self.now, i = heapq.heappop(ready)
            try:
                dt = next(warps[i])
                idle = idle + 1 if dt is None else 0
                if idle > 20000 and not self.events:
                    raise Fault("no warp gets on")
                heapq.heappush(ready, (self.now + (dt or self.rng.choice([1, 1, 3, 30])), i))
            except StopIteration:
                alive -= 1
        if self.in_flight:
            raise Fault("arrivals behind the end")


def kernel_of(seed, f8, **kw):
    rng = random.Random(seed)
    runs_a = [rng.choice([1, 2, 5, 13]) for _ in range(rng.choice([0, 0, 1, 2, 3]))]
    rows_a = rng.choice([(128, 128), (128, 1), (128, 64), (128, 90)])
    runs_b = [[(rng.choice([1, 1, 2, 3, 8]), rng.choice([1, 4, 7, 63, 64, 65, 128]))
               for _ in range(rng.choice([0, 1, 2, 5, 9]))] for _ in (0, 1)]
    return Kernel(rng, runs_a, rows_a, runs_b, f8, **kw)


@pytest.mark.parametrize("f8", [False, True], ids=["f16", "f8"])
def test_barriers(f8):
    for seed in range(150):
        kernel_of(seed, f8).run()


def test_one_barrier_for_both_slots_is_passed_early():
    faults = []
    for seed in range(60):
        try:
            kernel_of(seed, False, shared_full=True).run()
        except Fault as e:
            faults.append(str(e))
    assert any(f.startswith("passed early: full") for f in faults)
