"""The pages of a cache moved one by one on the host: what every operation on
the page table has to leave behind, whole number for whole number."""


class CacheOracle:
    """rows[slot]: the table row as a list of page indices (-1: given back)."""

    def __init__(self, n_slots, max_pages, n_pages, page):
        self.page, self.max_pages = page, max_pages
        self.rows = [[] for _ in range(n_slots)]
        self.lens, self.refs = [0] * n_slots, [0] * n_pages

    def _free(self):
        return [p for p, r in enumerate(self.refs) if r == 0]

    def _pages(self, n):
        return -(-n // self.page)

    def table(self):
        return [r + [-1] * (self.max_pages - len(r)) for r in self.rows]

    def extend(self, seqs, counts):
        """False, and nothing changed, where pages or columns do not suffice."""
        need = [self._pages(self.lens[s] + c) - self._pages(self.lens[s]) for s, c in zip(seqs, counts)]
        free = self._free()
        if sum(need) > len(free) or any(self._pages(self.lens[s] + c) > self.max_pages for s, c in zip(seqs, counts)):
            return False
        for s, c, n in zip(seqs, counts, need):
            for _ in range(n):
                self.rows[s].append(free.pop(0))
                self.refs[self.rows[s][-1]] = 1
            self.lens[s] += c
        return True

    def _drop(self, pages):
        for p in pages:
            if p >= 0:
                self.refs[p] -= 1

    def free(self, seqs):
        for s in seqs:
            self._drop(self.rows[s])
            self.rows[s], self.lens[s] = [], 0

    def trim(self, seqs, window, sinks):
        for s in seqs:
            for j, p in enumerate(self.rows[s]):
                if j * self.page >= sinks and (j + 1) * self.page <= self.lens[s] - window:
                    self._drop([p])
                    self.rows[s][j] = -1

    def fork(self, src, dst):
        """The copy list, or None with nothing changed."""
        free, copies, taken, new = self._free(), [], set(), []
        for s in src:
            row = list(self.rows[s])
            if self.lens[s] % self.page and (s not in dst or s in taken):
                if not free:
                    return None
                copies.append((row[-1], free.pop(0)))
                row[-1] = copies[-1][1]
            taken.add(s)
            new.append((row, self.lens[s]))
        for row, _ in new:
            for p in row:
                if p >= 0:
                    self.refs[p] += 1
        for d in dst:
            self._drop(self.rows[d])
        for d, (row, n) in zip(dst, new):
            self.rows[d], self.lens[d] = row, n
        return copies

    def compact(self):
        used = sum(r > 0 for r in self.refs)
        moves = list(zip([p for p in range(used, len(self.refs)) if self.refs[p]],
                         [p for p in range(used) if not self.refs[p]]))
        to = dict(moves)
        self.rows = [[to.get(p, p) for p in r] for r in self.rows]
        for a, b in moves:
            self.refs[b], self.refs[a] = self.refs[a], 0
        return moves
