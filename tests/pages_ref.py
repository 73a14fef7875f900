"""Plain reference of the calls on a page map (kt_page_map), one request after the other."""
from __future__ import annotations

BS = 128


def blocks_of(n):
    return -(-n // BS)


class Map:
    """Host copy of a page map; `bad` is set where a call records a device check."""

    def __init__(self, table, lens, blocks, refs):
        self.table = [list(map(int, row)) for row in table]
        self.lens, self.blocks = list(map(int, lens)), list(map(int, blocks))
        self.refs = list(map(int, refs))
        self.bad = False

    def lowest_free(self):
        return [p for p, r in enumerate(self.refs) if r <= 0]

    def check(self, ok):
        self.bad = self.bad or not ok
        return ok

    def free(self, seqs):
        for b in seqs:
            if not self.check(0 <= b < len(self.lens)):
                continue
            for p in self.table[b][: self.blocks[b]]:
                if self.check(0 <= p < len(self.refs)) and self.check(self.refs[p] > 0):
                    self.refs[p] -= 1
            self.lens[b] = self.blocks[b] = 0

    def fork(self, src, dst):
        """Returns the moves."""
        lens, blocks = list(self.lens), list(self.blocks)  # as they were before the call
        free, need, moves, taken = self.lowest_free(), 0, [], set()
        for s, d in zip(src, dst):
            ok = 0 <= s < len(lens) and 0 <= d < len(lens) and blocks[d] == 0 and lens[d] == 0
            ok = ok and 0 <= lens[s] <= BS * blocks[s] and blocks[s] <= len(self.table[s])
            if not self.check(ok and d not in taken):
                continue
            taken.add(d)
            n = lens[s]
            if n % BS:
                need += 1
                if not self.check(need <= len(free)):
                    continue
            if n == 0:
                continue
            for j in range(blocks_of(n)):
                p = self.table[s][j]
                self.check(0 <= p < len(self.refs))
                if n < (j + 1) * BS:
                    moves.append((p, free[need - 1]))
                    p = free[need - 1]
                    self.refs[p] = 1
                elif 0 <= p < len(self.refs):
                    self.refs[p] += 1
                self.table[d][j] = p
            self.lens[d], self.blocks[d] = n, blocks_of(n)
        return moves

    def reserve(self, more=None):
        free, at = self.lowest_free(), 0
        for b, n in enumerate(self.lens):
            m = 1 if more is None else more[b]
            if m == 0:
                continue
            width = len(self.table[b])
            want = blocks_of(n + m)
            if not self.check(m > 0 and n >= 0 and 0 <= self.blocks[b] <= width and want <= width):
                continue
            c = max(0, want - self.blocks[b])
            at += c
            if c and self.check(at <= len(free)):
                for i, p in enumerate(free[at - c:at]):
                    self.table[b][self.blocks[b] + i] = p
                    self.refs[p] = 1
                self.blocks[b] += c

    def compact(self):
        """Returns (moves, new table entries where a page is held else None, new counts)."""
        used = sum(r > 0 for r in self.refs)
        holes = [p for p in range(used) if self.refs[p] <= 0]
        moves = list(zip([p for p in range(used, len(self.refs)) if self.refs[p] > 0], holes))
        to = dict(moves)
        refs = [r if p < used else 0 for p, r in enumerate(self.refs)]
        for a, b in moves:
            refs[b] = self.refs[a]
        table = []
        for row, n in zip(self.table, self.blocks):
            self.check(0 <= n <= len(row))
            n = min(max(n, 0), len(row))
            for p in row[:n]:
                self.check(0 <= p < used or p in to)
            table.append([to.get(p, p) for p in row[:n]] + [None] * (len(row) - n))
        return moves, table, refs
