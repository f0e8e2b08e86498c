"""The oracle of the cache's page operations against what they are for: tokens
written page by page are read back, sequence by sequence, after any run of
operations, every page's count is the number of rows that hold it, and worked
examples come out as drawn by hand."""
import collections

import numpy as np
import pytest

import oracle


class Store:
    """The oracle with pages of tokens behind it and, beside them, each
    sequence's tokens as a plain list (None: given back)."""

    def __init__(self, *shape):
        self.o = oracle.CacheOracle(*shape)
        self.pages = [[None] * self.o.page for _ in self.o.refs]
        self.tokens = [[] for _ in self.o.rows]
        self.next = 0

    def extend(self, seqs, counts):
        if not self.o.extend(seqs, counts):
            return False
        for s, c in zip(seqs, counts):
            for _ in range(c):
                j = len(self.tokens[s])
                self.pages[self.o.rows[s][j // self.o.page]][j % self.o.page] = self.next
                self.tokens[s].append(self.next)
                self.next += 1
        return True

    def copy(self, moves):
        taken = [list(self.pages[a]) for a, _ in moves]
        for (_, b), x in zip(moves, taken):
            self.pages[b] = x

    def fork(self, src, dst):
        moves = self.o.fork(src, dst)
        if moves is None:
            return False
        self.copy(moves)
        new = [list(self.tokens[s]) for s in src]
        for d, x in zip(dst, new):
            self.tokens[d] = x
        return True

    def free(self, seqs):
        self.o.free(seqs)
        for s in seqs:
            self.tokens[s] = []

    def compact(self):
        self.copy(self.o.compact())
        used = sum(r > 0 for r in self.o.refs)
        assert all(self.o.refs[:used]) and not any(self.o.refs[used:])

    def check(self, gone):
        """`gone(s, j)`: whether token j of row s may have been given back."""
        o = self.o
        held = collections.Counter(p for row in o.rows for p in row if p >= 0)
        assert o.refs == [held[p] for p in range(len(o.refs))]
        for s, row in enumerate(o.rows):
            assert o.lens[s] == len(self.tokens[s]) and len(row) == -(-o.lens[s] // o.page) <= o.max_pages
            for j, t in enumerate(self.tokens[s]):
                page = row[j // o.page]
                if page < 0:
                    assert gone(s, j)
                else:
                    assert self.pages[page][j % o.page] == t
            # a page that is not full belongs to one sequence
            assert not (o.lens[s] % o.page and held[row[-1]] != 1)


@pytest.mark.parametrize("seed", range(8))
def test_tokens_survive_any_run_of_operations(seed):
    rng = np.random.default_rng(seed)
    n, window, sinks = 6, 21, 9
    c = Store(n, 12, 40, 8)
    trimmed = np.zeros(n, int)          # tokens of a row that a trim may have given back
    for _ in range(150):
        some = rng.permutation(n)[:rng.integers(1, n + 1)].tolist()
        what = rng.integers(6)
        if what <= 1:
            c.extend(some, rng.integers(0, 20, len(some)).tolist())
        elif what == 2:
            c.free(some[:2])
            trimmed[some[:2]] = 0
        elif what == 3:
            src = rng.integers(0, n, len(some)).tolist()
            if c.fork(src, some):
                trimmed[some] = trimmed[src]
        elif what == 4:
            c.o.trim(some, window, sinks)
            trimmed[some] = [max(trimmed[s], c.o.lens[s] - window) for s in some]
        else:
            c.compact()
        c.check(lambda s, j: sinks <= j < trimmed[s])


def test_an_extend_that_does_not_fit_changes_nothing():
    c = oracle.CacheOracle(2, 3, 4, 4)
    assert c.extend([0], [9]) and c.rows == [[0, 1, 2], []]
    before = (c.table(), list(c.lens), list(c.refs))
    assert not c.extend([1], [5])                 # one page is left, two are needed
    assert not c.extend([0], [4])                 # a fourth column
    assert (c.table(), c.lens, c.refs) == before
    assert c.extend([0, 1], [3, 4]) and c.rows == [[0, 1, 2], [3]]


def test_trim_gives_back_what_no_later_token_sees():
    for n in range(0, 40):
        for window in (1, 3, 4, 5, 11):
            for sinks in (0, 1, 4, 6):
                c = oracle.CacheOracle(1, 10, 10, 4)
                assert c.extend([0], [n])
                c.trim([0], window, sinks)
                i = n - 1                          # the earliest token still to ask
                seen = {j // 4 for j in range(n) if j > i - window or j < sinks}
                assert [p >= 0 for p in c.rows[0]] == [j in seen for j in range(len(c.rows[0]))]


def test_fork_and_compact_by_hand():
    c = oracle.CacheOracle(4, 3, 8, 4)
    assert c.extend([0, 1], [6, 4])               # row 0: pages 0 1 (half), row 1: page 2
    assert c.fork([0, 0, 1], [2, 3, 0]) == [(1, 3)]   # row 2, the first child of a replaced row, keeps page 1
    assert c.rows == [[2], [2], [0, 1], [0, 3]] and c.lens == [4, 4, 6, 6]
    assert c.refs == [2, 1, 2, 1, 0, 0, 0, 0] and c.compact() == []
    c.free([0, 1, 2])
    assert c.compact() == [(3, 1)] and c.rows[3] == [0, 1] and c.refs == [1, 1] + [0] * 6
    assert c.fork([3, 3], [0, 1]) == [(1, 2), (1, 3)]
    full = oracle.CacheOracle(2, 2, 1, 4)
    assert full.extend([0], [2]) and full.fork([0], [1]) is None and full.rows == [[0], []]
