"""The pages of a cache as include/libmtpspec/pages.h defines them, one row after another on the
host."""


class Pages:
    def __init__(self, B, wide, N, P):
        self.P, self.N, self.wide = P, N, wide
        self.table = [[-1] * wide for _ in range(B)]
        self.held, self.refs = [0] * B, [0] * N

    def take(self, b, n):
        """n further pages for row b, lowest first, to set a state up."""
        free = [p for p in range(self.N) if self.refs[p] == 0][:n]
        assert len(free) == n
        for p in free:
            self.hold(b, p)

    def hold(self, b, p):
        self.table[b][self.held[b]] = p
        self.held[b] += 1
        self.refs[p] += 1

    def drop(self, b, n):
        """Row b keeps n pages."""
        for i in range(n, self.held[b]):
            self.refs[self.table[b][i]] -= 1
            self.table[b][i] = -1
        self.held[b] = n

    def resize(self, keep, lens, copy=True):
        """(copies, whether there were too few pages, whether a length did not fit)."""
        P, B = self.P, len(self.held)
        fits = [k >= 0 and k <= self.held[b] * P and k <= n <= self.wide * P
                for b, (k, n) in enumerate(zip(keep, lens))]
        for b in range(B):
            if fits[b]:
                self.drop(b, -(-keep[b] // P))
        at = {}                                       # a partly filled last page's rows
        for b in range(B):
            if copy and fits[b] and keep[b] % P:
                at.setdefault(self.table[b][self.held[b] - 1], []).append(b)
        leaving = set()
        for p, rows in at.items():
            if self.refs[p] > 1:
                leaving |= set(rows[1:] if len(rows) == self.refs[p] else rows)
        free = [p for p in range(self.N) if self.refs[p] == 0]
        copies, short = [(-1, -1)] * B, False
        for b in range(B):
            grow = -(-lens[b] // P) - self.held[b] if fits[b] else 0
            n = grow + (b in leaving)
            if short or n > len(free):
                short = True
                continue
            new, free = free[:n], free[n:]
            if b in leaving:
                old = self.table[b][self.held[b] - 1]
                self.refs[old] -= 1
                self.table[b][self.held[b] - 1] = new[0]
                self.refs[new[0]] = 1
                copies[b] = (old, new.pop(0))
            for p in new:
                self.hold(b, p)
        wanting = any(fits[b] and self.held[b] < -(-lens[b] // P) for b in range(B)) or \
            any(copies[b] == (-1, -1) for b in leaving)
        return copies, wanting, any(not f and k >= 0 for f, k in zip(fits, keep))

    def fork(self, src, dst):
        bad = False
        for i, (s, d) in enumerate(zip(src, dst)):
            B = len(self.held)
            if not (0 <= s < B and 0 <= d < B) or s in dst or d in dst[i + 1:]:
                bad = True
                continue
            self.drop(d, 0)
            for p in self.table[s][:self.held[s]]:
                self.hold(d, p)
        return bad

    def compact(self):
        live = sum(r > 0 for r in self.refs)
        movers = [p for p in range(live, self.N) if self.refs[p] > 0]
        holes = [p for p in range(live) if self.refs[p] == 0]
        to = dict(zip(movers, holes))
        self.table = [[to.get(p, p) if i < self.held[b] else p for i, p in enumerate(t)]
                      for b, t in enumerate(self.table)]
        for a, b in to.items():
            self.refs[b], self.refs[a] = self.refs[a], 0
        return list(to.items())

    def agrees(self):
        """Whether the counts are those of the table, and no row holds a page twice."""
        count = [0] * self.N
        for b, t in enumerate(self.table):
            mine = t[:self.held[b]]
            assert len(set(mine)) == len(mine) and all(p == -1 for p in t[self.held[b]:])
            for p in mine:
                count[p] += 1
        return count == self.refs
